// Rotary positions of queries and keys.
//
// What it computes.  The first `rot` elements of each head are rot / 2 pairs; pair i of a row at position p is turned by the
// angle p f_i:
//     (a, b) -> amplitude * (a cos(p f_i) - b sin(p f_i), a sin(p f_i) + b cos(p f_i)),
// pairs being neighbours or a half of the turning part apart; the elements behind them stay as they are.
//
// Angles.  p f_i in fp32 is off by 0.06 at position 10^6.  What matters of it is the part of a turn that it ends on, so the
// frequency is held as a 64-bit fraction of a turn (2^64 f / 2 pi, mod 2^64): the product with an integer position, mod 2^64,
// is that part exactly, for positions of either sign, and what is lost is the fraction's own rounding: 2^-65 of a turn a position (2^-34 of
// one at the farthest), and 2^-52 of f for its quotient in double.
// The high bits as fp32 half-turns go to sincospif: an angle in [-pi, pi] off by at most 2^-24 of itself.
//
// How.  HBM bounds it (every element is read and written once), at a few rows the latency of one launch.  A unit is one access of
// 16 bytes (two, half a turning part apart, where pairs are halves) of a head.  A thread has one unit of the row, side after side, head
// after head, and takes it in several rows: where it is, is worked out once (unit by unit over rows and heads the divisions took
// longer than HBM: 16384 rows of 32 + 4 heads of 64 in fp16, half of each turning, took 48 us).  Threads load their first units, then make the
// block's cosines and sines, once for all heads, in shared memory, while those loads are on their way, and then store each two
// rows after the next two's loads (2 rows a block 32 us, 2 times 4 29.5: 5.1 TB/s; 32 + 8 heads of 128 in bf16 70 us: 4.8 TB/s).  Where sizes or
// addresses do not allow 16 bytes, accesses are of 8, 4 or of single elements.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/l2.h"
#include "l2_device.cuh"
#include "l2_rows.h"

namespace l2 {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;        // rows a thread takes at a time, where there are many
constexpr int kMostSteps = 4;   // so many times, the next rows loaded before the last are stored
constexpr int kBlocks = 6;      // blocks of an SM that more steps leave
constexpr int kTable = 2048;    // cosines and sines of a block
constexpr int kMaxAbreast = 16; // rows that lie side by side in a block

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

}  // namespace

template <typename T, int W, bool HALF, int K>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr bool kTwo = HALF || W == 1;  // a unit that turns is two accesses
    __shared__ float2 table[kTable];
    const int pairs = p.rot / 2;
    const int block = blockIdx.x / p.splits, part = blockIdx.x - block * p.splits;
    const int row0 = block * (p.abreast * K * p.steps), n_rows = min(p.abreast * K * p.steps, p.rows - row0);
    // the thread's unit, in rows `sub`, sub + abreast, ..
    const int sub = (int)((unsigned)threadIdx.x / (unsigned)p.part), u = part * p.part + threadIdx.x - sub * p.part;
    const int first = p.per_head[0] * p.s[0].heads;
    const bool second = u >= first, on = sub < p.abreast && u < p.units;
    const RopeSide &s = p.s[second];
    const int ph = p.per_head[second], v = second ? u - first : u, h = (int)((unsigned)v / (unsigned)ph), c = v - h * ph;
    // elements from a unit's first access to its second; units of a head that turn: W pairs each of halves, W elements of neighbours, one
    // pair where W is 1; behind them come the pieces that are copied
    const int apart = HALF ? pairs : 1;
    const int turning = HALF ? pairs / W : W == 1 ? pairs : p.rot / W;
    const bool turns = c < turning;
    const int e0 = turns ? (HALF ? c * W : W == 1 ? 2 * c : c * W) : p.rot + (c - turning) * W;
    const int pair = HALF ? c * W : W == 1 ? c : c * W / 2;
    const T *x = reinterpret_cast<const T *>(s.x + (row0 + sub) * s.x_row + h * s.x_head) + e0;
    T *y = reinterpret_cast<T *>(s.y + (row0 + sub) * s.y_row + h * s.y_head) + e0;
    const long long x_step = p.abreast * s.x_row / (long long)sizeof(T), y_step = p.abreast * s.y_row / (long long)sizeof(T);
    pdl_launch_dependents();
    pdl_wait();
    struct Step {  // K rows' units
        Piece<T, W> a[K], b[K];
    };
    auto load = [&](Step &x_, int step) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = step * K + k;
            if (!on || sub + i * p.abreast >= n_rows) continue;
            x_.a[k] = *reinterpret_cast<const Piece<T, W> *>(x + i * x_step);
            if (kTwo && turns) x_.b[k] = *reinterpret_cast<const Piece<T, W> *>(x + i * x_step + apart);
        }
    };
    Step now;
    load(now, 0);
    for (int i = threadIdx.x; i < n_rows * pairs; i += blockDim.x) {
        const int r = (int)((unsigned)i / (unsigned)pairs);
        const unsigned long long turn = (unsigned long long)(long long)p.positions[row0 + r] * p.turns[i - r * pairs];
        float sn, cs;
        sincospif((float)(long long)turn * 0x1p-63f, &sn, &cs);  // half-turns in [-1, 1]
        table[i] = make_float2(p.amplitude * cs, p.amplitude * sn);
    }
    __syncthreads();
#pragma unroll 1
    for (int step = 0;; ++step) {
        Step next;
        if (step + 1 < p.steps) load(next, step + 1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = step * K + k, r = sub + i * p.abreast;
            if (!on || r >= n_rows) continue;
            if (turns) {
                const float2 *t = table + r * pairs + pair;
                if constexpr (kTwo) {
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const float a = to_float(now.a[k].v[e]), b = to_float(now.b[k].v[e]);
                        now.a[k].v[e] = from_float<T>(a * t[e].x - b * t[e].y);
                        now.b[k].v[e] = from_float<T>(a * t[e].y + b * t[e].x);
                    }
                    *reinterpret_cast<Piece<T, W> *>(y + i * y_step + apart) = now.b[k];
                } else {
#pragma unroll
                    for (int e = 0; e < W / 2; ++e) {
                        const float a = to_float(now.a[k].v[2 * e]), b = to_float(now.a[k].v[2 * e + 1]);
                        now.a[k].v[2 * e] = from_float<T>(a * t[e].x - b * t[e].y);
                        now.a[k].v[2 * e + 1] = from_float<T>(a * t[e].y + b * t[e].x);
                    }
                }
            }
            *reinterpret_cast<Piece<T, W> *>(y + i * y_step) = now.a[k];
        }
        if (step + 1 >= p.steps) break;
        now = next;
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
    // a row's units over as few blocks as hold them, evenly; rows side by side where they are short
    p.splits = (p.units + kThreads - 1) / kThreads;
    p.part = (p.units + p.splits - 1) / p.splits;
    p.abreast = p.splits > 1 ? 1 : kThreads / p.part < kMaxAbreast ? kThreads / p.part : kMaxAbreast;
    // one row a thread while that leaves SMs without two blocks, then kRows at a time, as many times as leaves every SM kBlocks blocks
    const long long least = ((long long)p.rows + p.abreast - 1) / p.abreast * p.splits;
    const int k = least <= 2ll * num_sms ? 1 : kRows;
    while (p.abreast > 1 && p.abreast * k * pairs > kTable) --p.abreast;
    static_assert(kRows * kRopePairs <= kTable, "a block's rows have room for their cosines");
    const long long steps = least / ((long long)kBlocks * num_sms * k);
    p.steps = k == 1 || steps < 1 ? 1 : steps < kMostSteps ? (int)steps : kMostSteps;
    while (p.steps > 1 && p.abreast * k * p.steps * pairs > kTable) --p.steps;
    const int per = p.abreast * k * p.steps;
    const long long grid = ((long long)p.rows + per - 1) / per * p.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((p.part * p.abreast + 31) / 32 * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return k == 1 ? cudaLaunchKernelEx(&cfg, rope_kernel<T, W, HALF, 1>, p) : cudaLaunchKernelEx(&cfg, rope_kernel<T, W, HALF, kRows>, p);
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
