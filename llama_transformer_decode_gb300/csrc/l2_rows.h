// Operators on rows that a caller's own layer code makes: kernel parameter blocks and launch entry points (host side).
#pragma once
#include <cuda_runtime.h>

namespace l2 {

constexpr int kTreeNodes = 64;  // most drafted tokens of a sequence: one bit each of a 64-bit word

// Rotary positions (rope.cu).
constexpr int kRopePairs = 128;  // most pairs of a head that turn
struct RopeSide {                // queries, or keys
    const char *x;
    char *y;
    long long x_row, x_head, y_row, y_head;  // bytes
    int heads;
    int tail;                    // elements behind the turning ones to copy: 0 in place
};
struct RopeParams {
    RopeSide s[2];
    const int *positions;        // [rows]
    int rows, rot;
    float amplitude;
    // filled in by the launch
    int per_head[2];             // a head's units: pieces of `width` elements (or pairs) that turn, then pieces to copy
    int units;                   // of a row, both sides
    int splits, part, abreast;   // blocks of a row, units of each, rows side by side in one
    int steps;                   // times that a thread takes rows
    unsigned long long turns[kRopePairs];  // 2^64 times the turns that one position adds to each pair, mod 2^64
};
// half: pair i is elements i and i + rot / 2 (else 2 i and 2 i + 1); width: elements an access may take (1, 2, 4 or 8; at most
// 16 bytes), which the caller has found to divide every address and size.
cudaError_t launch_rope(RopeParams p, int dtype, bool half, int width, int num_sms, cudaStream_t s);

// Rules on logits (rules.cu): penalties, biases, masks.
struct RulesParams {
    const char *logits;          // [rows][vocab], rows in_row bytes apart
    char *out;
    long long in_row, out_row;   // bytes
    const int *seqs, *starts;    // [n] or nullptr (sequence i), [n + 1] or nullptr (one row each)
    const int *parents;          // [rows] or nullptr (chains)
    const int *drafted;          // [rows] tokens, or nullptr: no path counts
    const int *history;          // [n_seqs][history_stride]
    const int *lens, *counted;   // [n_seqs]; counted may be nullptr
    const float *repetition, *presence, *frequency;  // [n_seqs] or nullptr
    const int *bias_starts, *bias_tokens;            // [n_seqs + 1], [n_bias]
    const float *bias_values;
    const unsigned *masks;       // [n_masks][mask_stride] or nullptr
    const int *mask_rows;        // [rows] or nullptr (row r)
    int *err;
    long long history_stride, mask_stride;           // ints
    int vocab, rows, n, n_seqs, max_len, n_bias, n_masks;
    // filled in by the launch
    int slice, rows_per;         // tokens and rows of a block
};
// vec: elements an access (1 or 4, or 8 from 16 bits to 16 bits), which every row's address allows.
cudaError_t launch_rules(RulesParams p, int dtype, bool out_f32, int vec, int num_sms, cudaStream_t s);

}  // namespace l2
