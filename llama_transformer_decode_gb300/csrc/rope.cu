// Rotary positions of queries and keys.
//
// What it computes.  The first `rot` elements of each head are rot / 2 pairs; pair i of a row at position p is turned by the
// angle p f_i:
//     (a, b) -> amplitude * (a cos(p f_i) - b sin(p f_i), a sin(p f_i) + b cos(p f_i)),
// pairs being neighbours or a half of the turning part apart; the elements behind them stay as they are.
//
// Angles.  p f_i in fp32 is off by 0.06 at position 10^6.  What matters of it is the part of a turn that it ends on, so the
// frequency is held as a 64-bit fraction of a turn (2^64 f / 2 pi, mod 2^64): the product with an integer position, mod 2^64,
// is that part exactly, for positions of either sign, and the fraction's own rounding (2^-53 of f) is all that is lost.
// The high bits as fp32 half-turns go to sincospif: an angle in [-pi, pi] off by at most 2^-24 of itself.
//
// How.  HBM bounds it (every element is read and written once; 16384 rows of 32 + 4 heads of 64 in fp16: see the launch below), at a
// few rows the latency of one launch.  A unit is one access of 16 bytes (two, half a turning part apart, where pairs are
// halves), the whole head's, side after side.  A block takes the units of some rows, or a part of one row's; its
// threads load their units first, then make the rows' cosines and sines, once for all heads, in shared memory, while those
// loads are on their way.  Where sizes or addresses do not allow 16 bytes, accesses are of 8, 4 or of single elements.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/l2.h"
#include "l2_device.cuh"
#include "l2_rows.h"

namespace l2 {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;      // most units a thread holds
constexpr int kMaxRows = 16;   // most rows of a block

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// W elements moved as one access.
template <typename T, int W>
struct alignas(sizeof(T) * W) Piece {
    T v[W];
};

// Where a unit is: its first element in memory (and, in y, where it goes), its first pair, or -1 for one that is copied.
template <typename T>
struct Place {
    const T *x;
    T *y;
    int pair, row;  // row of the block's table
};

}  // namespace

template <typename T, int W, bool HALF, int K>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr bool kTwo = HALF || W == 1;  // a unit that turns is two accesses
    __shared__ float2 table[kMaxRows * kRopePairs];
    pdl_launch_dependents();
    pdl_wait();
    const int pairs = p.rot / 2;
    const int block = blockIdx.x / p.splits, part = blockIdx.x - block * p.splits;
    const int row0 = block * p.rows_per, n_rows = min(p.rows_per, p.rows - row0);
    // elements from a unit's first access to its second
    const int apart = HALF ? pairs : 1;
    // units of a head that turn: W pairs each of halves; W elements of neighbours, one pair where W is 1
    const int turning = HALF ? pairs / W : W == 1 ? pairs : p.rot / W;
    const int u0 = part * (K * kThreads), total = n_rows * p.units;
    auto place = [&](int u) {
        Place<T> a;
        a.row = (int)((unsigned)u / (unsigned)p.units);
        int v = u - a.row * p.units;
        const int first = p.per_head[0] * p.s[0].heads;
        const bool second = v >= first;
        if (second) v -= first;
        const RopeSide &s = p.s[second];
        const int ph = p.per_head[second], h = (int)((unsigned)v / (unsigned)ph), c = v - h * ph;
        const bool turns = c < turning;
        // first element: behind the turning part come the pieces that are copied
        const int e = turns ? (HALF ? c * W : W == 1 ? 2 * c : c * W) : p.rot + (c - turning) * W;
        a.x = reinterpret_cast<const T *>(s.x + (long long)(row0 + a.row) * s.x_row + h * s.x_head) + e;
        a.y = reinterpret_cast<T *>(s.y + (long long)(row0 + a.row) * s.y_row + h * s.y_head) + e;
        a.pair = !turns ? -1 : HALF ? c * W : W == 1 ? c : c * W / 2;
        return a;
    };
    Piece<T, W> xa[K], xb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int u = u0 + k * kThreads + threadIdx.x;
        if (u >= total) continue;
        const Place<T> a = place(u);
        xa[k] = *reinterpret_cast<const Piece<T, W> *>(a.x);
        if (kTwo && a.pair >= 0) xb[k] = *reinterpret_cast<const Piece<T, W> *>(a.x + apart);
    }
    // the rows' cosines and sines (a block that copies only would not need them: no such block is worth a test)
    for (int i = threadIdx.x; i < n_rows * pairs; i += kThreads) {
        const int r = i / pairs;
        const unsigned long long turn = (unsigned long long)(long long)p.positions[row0 + r] * p.turns[i - r * pairs];
        float sn, cs;
        sincospif((float)(long long)turn * 0x1p-63f, &sn, &cs);  // half-turns in [-1, 1]
        table[i] = make_float2(p.amplitude * cs, p.amplitude * sn);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int u = u0 + k * kThreads + threadIdx.x;
        if (u >= total) continue;
        const Place<T> a = place(u);
        if (a.pair >= 0) {
            const float2 *t = table + a.row * pairs + a.pair;
            if constexpr (kTwo) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float x = to_float(xa[k].v[e]), y = to_float(xb[k].v[e]);
                    xa[k].v[e] = from_float<T>(x * t[e].x - y * t[e].y);
                    xb[k].v[e] = from_float<T>(x * t[e].y + y * t[e].x);
                }
                *reinterpret_cast<Piece<T, W> *>(a.y + apart) = xb[k];
            } else {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                    const float x = to_float(xa[k].v[2 * e]), y = to_float(xa[k].v[2 * e + 1]);
                    xa[k].v[2 * e] = from_float<T>(x * t[e].x - y * t[e].y);
                    xa[k].v[2 * e + 1] = from_float<T>(x * t[e].y + y * t[e].x);
                }
            }
        }
        *reinterpret_cast<Piece<T, W> *>(a.y) = xa[k];
    }
}

namespace {

template <typename T, int W, bool HALF>
cudaError_t launch(RopeParams p, int num_sms, cudaStream_t s) {
    const int pairs = p.rot / 2, turning = HALF ? pairs / W : W == 1 ? pairs : p.rot / W;
    p.units = 0;
    for (int i = 0; i < 2; ++i) {
        p.per_head[i] = turning + p.s[i].tail / W;
        p.units += p.per_head[i] * p.s[i].heads;
    }
    if (p.units == 0) return cudaSuccess;
    // one unit a thread while that leaves SMs without a block, then up to kUnits: more loads in flight, and fewer cosines
    const long long blocks = ((long long)p.rows * p.units + kThreads - 1) / kThreads;
    const int k = blocks <= 2ll * num_sms ? 1 : kUnits;
    const int most = k * kThreads;
    p.rows_per = p.units >= most ? 1 : most / p.units < kMaxRows ? most / p.units : kMaxRows;
    p.splits = (p.units + most - 1) / most;
    const long long grid = ((long long)p.rows + p.rows_per - 1) / p.rows_per * p.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return k == 1 ? cudaLaunchKernelEx(&cfg, rope_kernel<T, W, HALF, 1>, p) : cudaLaunchKernelEx(&cfg, rope_kernel<T, W, HALF, kUnits>, p);
}

template <typename T>
cudaError_t launch(const RopeParams &p, bool half, int width, int num_sms, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (width == 8) return half ? launch<T, 8, true>(p, num_sms, s) : launch<T, 8, false>(p, num_sms, s);
    if (width >= 4) return half ? launch<T, 4, true>(p, num_sms, s) : launch<T, 4, false>(p, num_sms, s);
    if (width == 2) return half ? launch<T, 2, true>(p, num_sms, s) : launch<T, 2, false>(p, num_sms, s);
    return half ? launch<T, 1, true>(p, num_sms, s) : launch<T, 1, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int dtype, bool half, int width, int num_sms, cudaStream_t s) {
    if (dtype == L2_F32) return launch<float>(p, half, width, num_sms, s);
    if (dtype == L2_BF16) return launch<__nv_bfloat16>(p, half, width, num_sms, s);
    return launch<__half>(p, half, width, num_sms, s);
}

}  // namespace l2
