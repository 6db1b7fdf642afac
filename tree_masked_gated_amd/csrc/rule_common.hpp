// rule_common.hpp -- argument block, workspace layout and device helpers of the gated delta
// rule over whole sequences (internal to the library).
//
// The chunked form.  A chunk is kC = 64 rows of one sequence.  With H = S^T [d_k][d_v] the
// state before it, Gamma_i the sum of ln g over its rows up to i, a_i = e^Gamma_i and
// D_ij = e^(Gamma_i - Gamma_j):
//
//     L = strict_lower(D_ij k_i.k_j),   Y = lower(D_ij q_i.k_j)
//     F = V - a K H,   W = (I + L beta)^-1 F,   U = beta W    (row i of U is the write u_i of token i)
//     O = a Q H + Y U,                 H' = a_C H + sum_j e^(Gamma_C - Gamma_j) k_j u_j^T
//
// and, with dH' the gradient of H':
//
//     dU = Y^T dO + e^(Gamma_C - Gamma) K dH',   dR = (I + beta L)^-T dU,   dV = beta dR,   dbeta = dR . W
//     dH = a_C dH' + Q^T a dO - K^T a beta dR
//     dQ = a dO H^T + P K,  P = lower(D o dO U^T)
//     dK = P^T Q + (G + G^T) K + e^(Gamma_C - Gamma) U dH'^T - a beta dR H^T,
//                                                 G = strict_lower(-beta_i D_ij dR_i . U_j)
//     d ln g_t: over the paths that cross row t, as rule_join's comment says
//
// Both inverses come of one matrix, M = L (I + beta L)^-1: W = F - M (beta F) and
// dR = dU - M^T (beta dU).  The unit parts stay in fp32, and a beta of 0 needs no division.
//
// rule_prepare forms M and Y of all chunks at once; rule_scan, or rule_scan_wide for many slices, walks each
// sequence's chunks forward, a workgroup for a slice of the value columns; rule_scan_back
// walks them backward; rule_join forms dQ and dK of all chunks at once, and rule_gates
// the gates' gradients.
#pragma once

#include "attn_common.hpp"
#include "gdn_rule.h"
#include "mfma_tiles.hpp"
#include "rule_schedule.hpp"

namespace gdn {

struct RuleArgs {
    int B, Hk, Hv, group, dk, dv, n_slots;   // n_slots: chunk slots, T / kC + B
    int dvp;                                 // d_v rounded up to 32: row length of the workspace's value rows
    int64_t T;
    const int32_t* offsets;
    Rows q, k, v, o, d_o, dq, dk_out, dv_out; // strides in elements
    int vq, vk, vdo;                         // rows of q, k, d_o can be read 16 bytes at a time
    int vo;                                  // rows of o can be written 8 bytes at a time
    int direct;                              // the scan reads q and k from their rows
    const float* beta;
    const float* g;
    const float* S0;
    float* S_out;
    const float* dS_out;
    float* dS0;
    float* dbeta;
    float* dlog_g;
    char* kf; char* kt; char* qf; char* qt;  // operand fragments per (slot, key head)
    char* tm; char* tt; char* ym; char* yt;  // operand fragments per (slot, value head)
    float* coef;                             // per (slot, value head): a, e^(Gamma_C - Gamma), beta [3][kC]
    float* gram;                             // per (slot, key head): K K^T and Q K^T, tiles on and below the diagonal
    double* gam;                             // per (slot, value head): Gamma / ln 2 [kC]
    float* ht;                               // per (slot, value head): H [d_k padded][dvp]
    float* dht;                              // dH', the same layout
    float* w;                                // W [kC][dvp]
    float* dr;                               // dR [kC][dvp]
    float* pb; float* pe;                    // a slice's parts of dbeta and of d ln g's terms to the end [kC]
    float* pa;                               // parts of a_C <H, dH'>, of the rows of a slice's waves
    float* hs; float* zs;                    // rule_join's parts of d ln g: of h [kC], and sums of Z's tiles [2][10][16]
};

// Chunk slots.  Sequence b's chunks are slots base(b) .. , base(b) = offsets[b] / kC + b: the
// slots of different sequences never overlap and no table of them is needed.
__device__ __forceinline__ int slot_base(int64_t row0, int b) { return (int)(row0 / kC) + b; }

struct RuleSeq {
    int64_t row0;
    int n;                                   // rows, 0 for a sequence that cannot be used
};
__device__ __forceinline__ RuleSeq rule_seq(const RuleArgs& a, int b) {
    const int64_t o0 = a.offsets[b], o1 = a.offsets[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.T) return RuleSeq{0, 0};
    return RuleSeq{o0, (int)(o1 - o0)};
}

struct RuleChunk {
    int64_t row0;
    int n;                                   // rows of the chunk, 0: no chunk has this slot
};
// The chunk of a slot: every lane looks at one sequence, 64 at a time.
__device__ __forceinline__ RuleChunk rule_chunk(const RuleArgs& a, int slot) {
    const int lane = threadIdx.x & 63;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        bool mine = false;
        RuleSeq s{0, 0};
        if (b < a.B) {
            s = rule_seq(a, b);
            const int base = slot_base(s.row0, b);
            mine = s.n > 0 && slot >= base && slot - base < (s.n + kC - 1) / kC;
        }
        const uint64_t m = __ballot(mine);
        if (m) {
            const int src = __ffsll((unsigned long long)m) - 1;
            const int row0 = __shfl((int)s.row0, src), n = __shfl(s.n, src);
            const int at = (slot - slot_base(row0, b0 + src)) * kC;
            return RuleChunk{(int64_t)row0 + at, min(kC, n - at)};
        }
    }
    return RuleChunk{0, 0};
}

// Fragments that a lower (upper) triangular 64 x 64 operand needs: row tile i, 32-wide step s.
__host__ __device__ constexpr int low_frag(int i, int s) { return i < 2 ? i : 2 + 2 * (i - 2) + s; }
__host__ __device__ constexpr int up_frag(int i, int s) { return i < 2 ? 2 * i + s : 2 + i; }
constexpr int kTriFrags = 6;
constexpr int kFrag = 64 * 16;               // bytes of one fragment: 16 per lane

// p the same for the wave: the lane's part of the address is a 32-bit offset of its own.
__device__ __forceinline__ bf16x8 load_frag(const char* p, int lane) {
    return *reinterpret_cast<const bf16x8*>(p + (uint32_t)(lane * 16));
}
__device__ __forceinline__ void store_frag(char* p, int lane, bf16x8 x) {
    *reinterpret_cast<bf16x8*>(p + lane * 16) = x;
}

// Factors of the matrix products, as sums of bf16 terms.  A bf16 element is one term.  An fp32
// factor is three (24 bits) wherever the product reaches a state, a gate's gradient or an fp32
// row: two would leave 2^-18 per factor, several 1e-6 at the end of a chunk.  Products that only
// reach bf16 rows take two terms of it.
template <int IO>
constexpr int kPlanes = IO == GDN_BF16 ? 1 : 3;      // an io element
constexpr int kSum = 3;                              // an fp32 factor
template <int IO>
constexpr int kRound = IO == GDN_BF16 ? 2 : 3;       // an fp32 factor of a product for io rows alone

// Two values as the next term of each, packed; what is left of them stays in x and y.
__device__ __forceinline__ uint32_t next_term(float& x, float& y, bool last) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t t = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
    if (!last) {
        x -= __uint_as_float(t << 16);
        y -= __uint_as_float(t & 0xffff0000u);
    }
    return t;
}
template <int P>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&to)[P]) {
    u32x4 t[P];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float u = x[2 * j], v = x[2 * j + 1];
#pragma unroll
        for (int p = 0; p < P; ++p) t[p][j] = next_term(u, v, p == P - 1);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) to[p] = __builtin_bit_cast(bf16x8, t[p]);
}
template <int P>
__device__ __forceinline__ void split4p(f32x4 x, s16x4 (&to)[P]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x2 t[P];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float u = x[2 * j], v = x[2 * j + 1];
#pragma unroll
        for (int p = 0; p < P; ++p) t[p][j] = next_term(u, v, p == P - 1);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) to[p] = __builtin_bit_cast(s16x4, t[p]);
}

// An io element, rounded to nearest.
template <int IO>
__device__ __forceinline__ void put_io(char* p, int64_t i, float x) {
    if constexpr (IO == GDN_BF16)
        reinterpret_cast<uint16_t*>(p)[i] = bf16_rne(x);
    else
        reinterpret_cast<float*>(p)[i] = x;
}

template <int IO>
struct Planes {
    bf16x8 p[kPlanes<IO>];
};

// Columns col .. col + 7 of a row of d elements as operand planes, zeros past d and where !live.
template <int IO>
__device__ __forceinline__ Planes<IO> load_row8(const char* base, int64_t at, int col, int d, bool vec, bool live) {
    Planes<IO> r;
    if constexpr (IO == GDN_BF16) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at + col;
        bf16x8 x;
        if (vec) {
            const u32x4 z = {0, 0, 0, 0};
            x = __builtin_bit_cast(bf16x8, live && col < d ? *reinterpret_cast<const u32x4*>(p) : z);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __builtin_bit_cast(__bf16, live && col + j < d ? p[j] : (uint16_t)0);
        }
        r.p[0] = x;
    } else {
        const float* p = reinterpret_cast<const float*>(base) + at + col;
        float x[8];
        if (vec) {
            const f32x4 z = {0, 0, 0, 0};
            const bool in = live && col < d;
            const f32x4 u = in ? *reinterpret_cast<const f32x4*>(p) : z;
            const f32x4 w = in ? *reinterpret_cast<const f32x4*>(p + 4) : z;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = u[j], x[4 + j] = w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = live && col + j < d ? p[j] : 0.f;
        }
        split8(x, r.p);
    }
    return r;
}

// acc += A B over the pairs of terms that matter: with the most terms of a factor n, those whose
// orders sum to less than n.
template <int PA, int PB, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 acc) {
    static_assert(PA <= NA && PB <= NB, "terms");
    constexpr int n = PA > PB ? PA : PB;
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
        for (int j = 0; j < PB; ++j)
            if (i + j < n) acc = mfma32(a[i], b[j], acc);
    return acc;
}

// Four rows of an accumulator column, as bf16 terms, to a [column][row] tile in LDS.
template <int P>
__device__ __forceinline__ void put4(uint16_t* at, int plane, f32x4 x) {
    s16x4 t[P];
    split4p(x, t);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<s16x4*>(at + p * plane) = t[p];
}
template <int P>
__device__ __forceinline__ void get8(const uint16_t* at, int plane, bf16x8 (&x)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = *reinterpret_cast<const bf16x8*>(at + p * plane);
}

template <int IO, int DK>
hipError_t rule_forward_launch(const RuleArgs& a, hipStream_t stream);
template <int IO, int DK>
hipError_t rule_backward_launch(const RuleArgs& a, hipStream_t stream);

struct RuleStepArgs {
    int B, Hk, Hv, group, dk, dv, n_states;
    const int32_t* slot;
    Rows q, k, v, o;
    const float* beta;
    const float* g;
    float* state;
};
hipError_t launch_rule_step(const RuleStepArgs& a, int io, hipStream_t stream);

}  // namespace gdn
