// rule_kernels.hpp -- the chunked gated delta rule on MFMA (see rule_common.hpp for the
// mathematics), compiled for one element type and padded d_k per source file.
#pragma once

#include "rule_common.hpp"

namespace gdn {

// Rows of the LDS tiles are padded by 8 elements: 16-byte reads of 16 rows then spread over all banks.
constexpr int kTp = kC + 8;

// ------------------------------------------------------------------ prepare
//
// One workgroup of four waves per (chunk slot, key head).  Wave w owns row tile w (16 rows).
// The chunk's keys and queries are laid out as matrix operands once, for every value head and
// slice that reads them; the products K K^T and Q K^T are formed once per key head, and each of
// its value heads makes its M and Y of them.  M is formed in fp32 (diagonal blocks by
// substitution, the others by fp32 matrix instructions) and kept as bf16 terms.
//
// Bound by what it writes: 8192 rows of 16 / 32 heads of 128, bf16, 84 us for 230 MB written and 62
// MB read; 25331 rows in 24 sequences, without K's and Q's operands, 181 us for 518 and 183 MB.
template <int IO, int DK, bool BACK>
__global__ void __launch_bounds__(256) rule_prepare(const RuleArgs a) {
    constexpr int P = kPlanes<IO>, R = kRound<IO>, KS = DK / 32, NT = DK / 16, LD = DK + 8;
    constexpr int TP = kC + 4;                       // fp32 row, whole 16-byte pieces
    __shared__ __attribute__((aligned(16))) uint16_t rows[P][kC][LD];
    __shared__ __attribute__((aligned(16))) float xs[kC][TP];
    __shared__ __attribute__((aligned(16))) float ts[kC][TP];
    __shared__ double gam[kC];
    __shared__ __attribute__((aligned(16))) float bet[kC];

    const int slot = blockIdx.x, hk = blockIdx.y;
    const RuleChunk ch = rule_chunk(a, slot);
    if (ch.n == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const int row = 16 * wv + n;                     // this lane's row of an operand tile
    const bool live = row < ch.n;
    const int64_t grow = ch.row0 + (live ? row : 0);
    const size_t key = (size_t)slot * a.Hk + hk;
    constexpr size_t kTile = (size_t)P * 4 * KS * kFrag;

    // K: operand fragments of its rows, and the rows in LDS
    Planes<IO> kfr[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        kfr[s] = load_row8<IO>(a.k.p, grow * a.k.row + (int64_t)hk * a.k.head, 32 * s + 8 * q4, a.dk, a.vk, live);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!a.direct) store_frag(a.kf + key * kTile + ((p * 4 + wv) * KS + s) * kFrag, lane, kfr[s].p[p]);
            *reinterpret_cast<bf16x8*>(&rows[p][row][32 * s + 8 * q4]) = kfr[s].p[p];
        }
    }
    Planes<IO> qfr[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qfr[s] = load_row8<IO>(a.q.p, grow * a.q.row + (int64_t)hk * a.q.head, 32 * s + 8 * q4, a.dk, a.vq, live);
        if (!BACK && !a.direct)
#pragma unroll
            for (int p = 0; p < P; ++p)
                store_frag(a.qf + key * kTile + ((p * 4 + wv) * KS + s) * kFrag, lane, qfr[s].p[p]);
    }
    __syncthreads();
    // the lower row tiles of K K^T and Q K^T
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        kk[j] = qk[j] = f32x4{0, 0, 0, 0};
        if (j > wv) continue;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            bf16x8 b[P];
            get8<P>(&rows[0][16 * j + n][32 * s + 8 * q4], kC * LD, b);
            kk[j] = mma<P, P>(kfr[s].p, b, kk[j]);
            qk[j] = mma<P, P>(qfr[s].p, b, qk[j]);
        }
    }
    if constexpr (BACK)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wv) {
                f32x4* to = reinterpret_cast<f32x4*>(a.gram) + (((size_t)slot * a.Hk + hk) * 10 + wv * (wv + 1) / 2 + j) * 128;
                to[lane] = kk[j];
                to[64 + lane] = qk[j];
            }
    // transposed operands: 8 rows of one column per lane
    auto transposed = [&](char* to) {
        for (int t = wv; t < NT; t += 4)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    bf16x8 x;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = __builtin_bit_cast(__bf16, rows[p][32 * s + 8 * q4 + j][16 * t + n]);
                    store_frag(to + key * kTile + ((p * NT + t) * 2 + s) * kFrag, lane, x);
                }
    };
    transposed(a.kt);
    if constexpr (BACK) {
        __syncthreads();
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<bf16x8*>(&rows[p][row][32 * s + 8 * q4]) = qfr[s].p[p];
        __syncthreads();
        transposed(a.qt);
    }

    // fragments of a lower triangular tile, and of its transpose
    auto keep = [&](const float (&v)[8], char* to, int f, auto planes) {
        bf16x8 x[decltype(planes)::value];
        split8(v, x);
#pragma unroll
        for (int p = 0; p < decltype(planes)::value; ++p) store_frag(to + (f * decltype(planes)::value + p) * kFrag, lane, x[p]);
    };
    auto low = [&](const float (*x)[TP], char* to, auto planes) {
        for (int f = wv; f < kTriFrags; f += 4) {
            const int i = f < 2 ? f : 2 + (f - 2) / 2, s = f < 2 ? 0 : (f - 2) % 2;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[16 * i + n][32 * s + 8 * q4 + j];
            keep(v, to, f, planes);
        }
    };
    auto up = [&](const float (*x)[TP], char* to) {
        for (int f = wv; f < kTriFrags; f += 4) {
            const int i = f < 4 ? f / 2 : f - 2, s = f < 4 ? f % 2 : 1;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[32 * s + 8 * q4 + j][16 * i + n];
            keep(v, to, f, std::integral_constant<int, kSum>());
        }
    };

    for (int gi = 0; gi < a.group; ++gi) {
        const int hv = hk * a.group + gi;
        const size_t val = (size_t)slot * a.Hv + hv;
        if (wv == 0) {                               // running sums of log2 g, in fp64
            const bool in = lane < ch.n;
            const int64_t at = (ch.row0 + (in ? lane : 0)) * a.Hv + hv;
            const float b = in ? a.beta[at] : 0.f;
            // A gate of 0: differences across it have no power of 2 in fp32, others keep theirs.
            const float g = a.g[at];
            double x = !in ? 0.0 : g == 0.f ? -1000.0 : (double)log2f(g);
#pragma unroll
            for (int off = 1; off < 64; off *= 2) {
                const double y = __shfl_up(x, off);
                if (lane >= off) x += y;
            }
            gam[lane] = x;
            bet[lane] = b;
            float* c = a.coef + val * 3 * kC;
            c[lane] = exp2f((float)x);
            c[kC + lane] = exp2f((float)(__shfl(x, 63) - x));
            c[2 * kC + lane] = b;
            if constexpr (BACK) a.gam[val * kC + lane] = x;
        }
        __syncthreads();
        // Y to ts, L to xs: this wave's row tile; the tile right of an even diagonal one is zero
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > (wv | 1)) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * wv + 4 * q4 + r, c = 16 * j + n;
                const float d = c <= i ? exp2f((float)(gam[i] - gam[c])) : 0.f;
                ts[i][c] = c <= i ? d * qk[j][r] : 0.f;
                xs[i][c] = c < i ? d * kk[j][r] : 0.f;
            }
        }
        __syncthreads();
        if constexpr (BACK)
            up(ts, a.yt + val * kSum * kTriFrags * kFrag);
        else
            low(ts, a.ym + val * R * kTriFrags * kFrag, std::integral_constant<int, R>());
        __syncthreads();
        // M's diagonal blocks, row by row: M_i = sum_(j<i) L_ij T_j, T_i = e_i - beta_i M_i; lane
        // (n, q) has column n of block q
        if (wv == 0) {
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float m = 0.f;
#pragma unroll
                for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(&xs[16 * q4 + i][16 * q4 + 4 * j4]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (4 * j4 + j < i) m += x[j] * t[4 * j4 + j];
                }
                t[i] = (i == n ? 1.f : 0.f) - bet[16 * q4 + i] * m;
                ts[16 * q4 + i][16 * q4 + n] = m;
            }
        }
        __syncthreads();
        // the blocks below, a block diagonal at a time: with A = sum_(j<=k<i) L_ik T_kj,
        // M_ij = (I - M_ii beta) A.  Contraction step r of a 16 x 16 product takes indexes
        // 4 q + r, which is how accumulators lie.
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            if (wv >= d) {
                const int j = wv - d;
                f32x4 acc = {0, 0, 0, 0};
                for (int k = j; k < wv; ++k) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(&xs[row][16 * k + 4 * q4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int kk_ = 4 * q4 + r;
                        const float t = (k == j && kk_ == n ? 1.f : 0.f) - bet[16 * k + kk_] * ts[16 * k + kk_][16 * j + n];
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], t, acc, 0, 0, 0);
                    }
                }
                const f32x4 m = *reinterpret_cast<const f32x4*>(&ts[row][16 * wv + 4 * q4]);
                f32x4 out = acc;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    out = __builtin_amdgcn_mfma_f32_16x16x4f32(-m[r], bet[16 * wv + 4 * q4 + r] * acc[r], out, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) ts[16 * wv + 4 * q4 + r][16 * j + n] = out[r];
            }
            __syncthreads();
        }
        low(ts, a.tm + val * kSum * kTriFrags * kFrag, std::integral_constant<int, kSum>());
        if constexpr (BACK) up(ts, a.tt + val * kSum * kTriFrags * kFrag);
        __syncthreads();
    }
}

// A [row][column] tile of 16 columns in LDS, as operands of 32-row contraction steps: step k holds
// lane l's eight rows 32 k + 8 (l / 16) .. of column l % 16 at l * 8.  place4: rows row .. row + 3, row a
// multiple of 4, of a tile that begins with step `first`.
constexpr int kStep = 64 * 8;
__device__ __forceinline__ int place4(int first, int row, int n) {
    return ((first + (row >> 5)) * 64 + n + 16 * ((row >> 3) & 3)) * 8 + (row & 4);
}

// Nothing is moved past this: operands that are read before it are on their way during what follows,
// where the compiler would read each just before its use and wait for it.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

// The place-th longest sequence, where there are more workgroups than places for them: those that
// take longest begin first, so that none begins when the rest are nearly done.  A wave orders up to
// 64 sequences by itself; with more, what a place gets averages out.  (24 prompts of 0 to 2048 rows,
// 32 heads, wide scan: 505 us in the order of the batch, 443 longest first.)
constexpr int kPlaces = 512;                         // two workgroups to a compute unit
__device__ __forceinline__ int longest(const RuleArgs& a, int place) {
    if (gridDim.x <= kPlaces || a.B > 64) return place;
    const int lane = threadIdx.x & 63;
    const int n = lane < a.B ? rule_seq(a, lane).n : -1;
    int before = 0;
    for (int j = 0; j < a.B; ++j) {
        const int other = __builtin_amdgcn_readlane(n, j);
        before += other > n || (other == n && j < lane);
    }
    return __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(lane < a.B && before == place)) - 1);
}

template <int IO, int DK>
__device__ __forceinline__ void scan_place(const RuleArgs& a, int slices, int& b, int& hv, int& sl) {
    // Workgroups go to the eight XCDs in turn: the slices of a head stay on one, whose L2 they share.
    const int heads = a.B * a.Hv, blk = blockIdx.x;
    const int whole = heads / 8 * 8 * slices;
    int head;
    if (blk < whole) {
        head = blk / (8 * slices) * 8 + blk % 8;
        sl = blk / 8 % slices;
    } else {
        head = heads / 8 * 8 + (blk - whole) / slices;
        sl = (blk - whole) % slices;
    }
    b = head / a.Hv;
    hv = head - b * a.Hv;
    b = longest(a, b);
}


// Elements of value rows, four rows 16 i + 4 q4 + r of a chunk in one column: requested a chunk
// ahead as they lie in memory, converted and masked where they are used, so that nothing waits for
// them before.  A lane's four places are kept as offsets from the chunk's first row; the last
// chunk's rows past the sequence's end are read from its last row.
template <int IO>
struct Rows4 {
    typedef std::conditional_t<IO == GDN_BF16, uint16_t, float> E;
    const E* at;                                     // column of the chunk's first row
    int64_t step;                                    // a chunk's rows
    int64_t off[4];
    E x[4];
    int row;                                         // of the chunk
    bool in;                                         // a column of the tensor
    __device__ __forceinline__ void begin(const Rows& from, int64_t row0, int64_t head, int row_, int col, int d) {
        at = reinterpret_cast<const E*>(from.p) + row0 * from.row + head + min(col, d - 1);
        step = kC * from.row;
        row = row_;
        in = col < d;
#pragma unroll
        for (int r = 0; r < 4; ++r) off[r] = (row + r) * from.row;
    }
    // the places of a chunk of `rows` rows
    __device__ __forceinline__ void places(int64_t stride, int rows) {
#pragma unroll
        for (int r = 0; r < 4; ++r) off[r] = row_in(row + r, rows) * stride;
    }
    __device__ __forceinline__ void load(int64_t chunk) {
        const E* p = at + chunk * step;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = p[off[r]];
    }
    __device__ __forceinline__ f32x4 get(int rows) const {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float y;
            if constexpr (IO == GDN_BF16) y = bf16_bits_to_f32(x[r]); else y = x[r];
            v[r] = in && row + r < rows ? y : 0.f;
        }
        return v;
    }
};

// Which row tiles and columns of a slice a wave works on: items x < kItems of the wave's row tiles
// ii < NI.  With eight waves the two halves take one column block each.
template <int NW, int NC>
struct Deal {
    static_assert(NW <= 4 || NC == 2, "eight waves share two column blocks");
    static constexpr int NI = NW < 4 ? 4 / NW : 1;
    static constexpr int NX = NW <= 4 ? NC : 1;      // column blocks of a wave
    int wv;
    __device__ int tile(int ii) const { return NW <= 4 ? wv + ii * NW : wv & 3; }
    __device__ int block(int x) const { return NW <= 4 ? x : wv >> 2; }
};

// The outputs' part of a scan: O = a Q H + Y U of some row tiles and column blocks.  Its operands are
// held and requested like the state's.
template <int IO, int DK, int NI, int NX>
struct Outputs {
    static constexpr int P = kPlanes<IO>, R = kRound<IO>, KS = DK / 32;
    static constexpr bool kHold = DK * P <= 256;
    bf16x8 qf[NI][kHold ? KS : 1][P], ym[NI][2][R];
    f32x4 ca[NI], o[NI][NX];
    const char *pq, *py;
    const float* pc;
    int64_t off[NI][4];                              // this lane's rows of a chunk of o
    int tile[NI];

    __device__ __forceinline__ void begin(const RuleArgs& a, size_t key, size_t val, int lane) {
        pq = a.qf + key;
        py = a.ym + val * R * kTriFrags * kFrag;
        pc = a.coef + val * 3 * kC;
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int r = 0; r < 4; ++r) off[ii][r] = (16 * tile[ii] + 4 * (lane >> 4) + r) * a.o.row;
    }
    __device__ __forceinline__ void load_step(int s, int to, int lane) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int p = 0; p < P; ++p) qf[ii][to][p] = load_frag(pq + ((p * 4 + tile[ii]) * KS + s) * kFrag, lane);
    }
    __device__ __forceinline__ void load_q(int lane) {
        if constexpr (kHold)
#pragma unroll
            for (int s = 0; s < KS; ++s) load_step(s, s, lane);
    }
    __device__ __forceinline__ void load_y(int lane) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            ca[ii] = *reinterpret_cast<const f32x4*>(pc + 16 * tile[ii] + 4 * (lane >> 4));
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < R; ++p)
                    ym[ii][s][p] = load_frag(py + (low_frag(tile[ii], min(s, tile[ii] / 2)) * R + p) * kFrag, lane);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) o[ii][x] = f32x4{0, 0, 0, 0};
    }
    // += Q H for one contraction step and column block; hb: that step of H
    template <int N>
    __device__ __forceinline__ void add(int s, int x, const bf16x8 (&hb)[N]) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) o[ii][x] = mma<P, R>(qf[ii][kHold ? s : 0], hb, o[ii][x]);
    }
    // u: the column block's tile of U; to: the chunk's first row of o, this lane's column
    __device__ __forceinline__ void finish(int x, const uint16_t* u, int plane, char* to, int rows, bool in, int lane) {
        const int q4 = lane >> 4;
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            f32x4 y = ca[ii] * o[ii][x];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s > tile[ii] / 2) continue;
                bf16x8 ub[R];
                get8<R>(u + s * kStep + lane * 8, plane, ub);
                y = mma<R, R>(ym[ii][s], ub, y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (in && 16 * tile[ii] + 4 * q4 + r < rows) put_io<IO>(to, off[ii][r], y[r]);
        }
    }
};

// Waves of the outputs, where they have their own.
template <int DK>
constexpr int kOutWaves = DK / 32 < 4 ? DK / 32 : 4;

// OUT: what becomes of the outputs.
enum { kOutNone = 0, kOutOwn = 1, kOutSame = 2 };    // not formed; by waves of their own; by the state's waves

// ------------------------------------------------------------------ scan
//
// One workgroup per (sequence, value head, slice of 16 NC value columns).  d_k / 32 state waves:
// wave w keeps rows 32 w .. 32 w + 31 of the slice of H in accumulators (fp32).  A chunk goes in four
// phases with a barrier between them: every wave's H goes to LDS as operand terms; row tile i (16
// rows) of K H, then of W, is formed by wave i, which needs all of the one before; H' needs all of
// U.  The outputs are formed by waves of their own, from the terms of H and U that the state waves
// leave in LDS, in the time that those take for the next step.  Terms lie in LDS as operands are
// read, 16 bytes to a lane (rows padded to spread over the banks took twice the reads' time);
// accumulators have four rows to a lane, 8 bytes of that.  (Parts of K H from each wave's own rows
// of H, added up in LDS, took 1.1 times as long: 16-byte LDS writes take 20 to 40 cycles each where
// reads take 9.)
//
// A single sequence's scan is bound by what one state wave issues per chunk, one after the other,
// so addresses are kept as running pointers, and operands of a chunk are requested while the chunk
// before it is worked on.  8192 rows, 32 heads of 128, bf16: 248 us, 1.9 us a chunk; the
// matrix units are busy for 18 % of it, waves wait for 55 % of their time, for the phases' LDS writes, barriers
// and reads.
// BACK: instead of the outputs, the state before each chunk and W are kept for the gradients.
template <int IO, int DK, int NC, int OUT>
__global__ void __launch_bounds__(DK * 2 + (OUT == kOutOwn ? 64 * kOutWaves<DK> : 0), IO == GDN_BF16 && DK == 128 ? 2 : 1)
rule_scan(const RuleArgs a) {
    constexpr int P = kPlanes<IO>, KS = DK / 32, NW = KS, NT = DK / 16;
    constexpr int S = kSum, R = kRound<IO>;
    constexpr bool BACK = OUT == kOutNone;
    typedef Deal<NW, NC> D;
    constexpr int NI = D::NI, NX = D::NX;
    constexpr bool kHold = DK * P <= 256;            // K and Q are held in registers, or read as they are used
    constexpr int KH = kHold ? KS : 1;
    constexpr int kPl = NC * 2 * kStep, kPh = NC * KS * kStep; // elements of a term of a tile
    __shared__ __attribute__((aligned(16))) uint16_t hh[S * kPh], rr[S * kPl], uu[R * kPl], ue[S * kPl];

    int b, hv, sl;
    scan_place<IO, DK>(a, a.dvp / (16 * NC), b, hv, sl);
    const int hk = hv / a.group;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const RuleSeq seq = rule_seq(a, b);
    const int chunks = chunks_of(seq.n), base = slot_base(seq.row0, b);
    const int tail = last_rows(seq.n);          // rows of the last chunk
    const int col0 = sl * 16 * NC + n;               // this lane's columns: col0 + 16 c
    constexpr size_t kTile = (size_t)P * 4 * KS * kFrag;
    constexpr size_t kTri = (size_t)kTriFrags * kFrag;
    const size_t key = ((size_t)base * a.Hk + hk) * kTile, val = (size_t)base * a.Hv + hv;
    const size_t key_step = (size_t)a.Hk * kTile, y_step = (size_t)a.Hv * R * kTri;
    const float* co = a.coef + val * 3 * kC;         // of the chunk that is worked on
    const size_t co_step = (size_t)a.Hv * 3 * kC;
    constexpr int E = IO == GDN_BF16 ? 2 : 4;
    char* po = OUT == kOutNone ? nullptr : a.o.p + (seq.row0 * a.o.row + hv * a.o.head + col0) * E;
    const int64_t o_step = kC * a.o.row * E;

    if (OUT == kOutOwn && wv >= NW) {
        constexpr int OW = kOutWaves<DK>, OI = 4 / OW;
        Outputs<IO, DK, OI, NC> out;
#pragma unroll
        for (int ii = 0; ii < OI; ++ii) out.tile[ii] = wv - NW + ii * OW;
        out.begin(a, key, val, lane);
        if (chunks > 0) {
            out.load_q(lane);
            out.load_y(lane);
        }
        for (int c = 0; c < chunks; ++c) {
            const bool more = c + 1 < chunks;
            out.clear();
            lds_barrier();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if constexpr (!kHold) out.load_step(s, 0, lane);
#pragma unroll
                for (int cc = 0; cc < NC; ++cc) {
                    bf16x8 hb[R];
                    get8<R>(hh + (cc * KS + s) * kStep + lane * 8, kPh, hb);
                    out.add(s, cc, hb);
                }
            }
            out.pq += more ? key_step : 0;
            out.load_q(lane);
            lds_barrier();
            lds_barrier();
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
                out.finish(cc, uu + 2 * cc * kStep, kPl, po + 16 * cc * E, more ? kC : tail, col0 + 16 * cc < a.dv, lane);
            po += o_step;
            out.py += more ? y_step : 0;
            out.pc += more ? co_step : 0;
            out.load_y(lane);
        }
        return;
    }

    // ---- the state
    const D deal{wv};
    if constexpr (OUT == kOutOwn) __builtin_amdgcn_s_setprio(2); // the outputs' waves fill in
    // H: rows 32 wv + 16 t + 4 q4 + r, columns col0 + 16 c
    f32x4 h[2][NC];
    const size_t state = ((size_t)b * a.Hv + hv) * a.dv * a.dk;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 32 * wv + 16 * t + 4 * q4 + r, j = col0 + 16 * c;
                h[t][c][r] = a.S0 && i < a.dk && j < a.dv ? a.S0[state + (size_t)j * a.dk + i] : 0.f;
            }

    // The operands of a chunk are requested for the next one as soon as they have been used.  No
    // request is conditional: the compiler could not count the ones in flight, and would wait for all.
    bf16x8 kf[NI][KH][P], tm[NI][2][S], kt[2][2][P];
    f32x4 ca[NI], ce[NI], cb[NI];
    Rows4<IO> v[NI][NX];
    Outputs<IO, DK, NI, NX> out;                     // kOutSame
    float end;
    const char* pk = a.kf + key;
    const char* pt = a.kt + key + 2 * wv * 2 * kFrag;
    const char* pm = a.tm + val * S * kTri;
    const size_t m_step = (size_t)a.Hv * S * kTri;
    const float *pca = co, *pcb = co;
    float* ph = BACK ? a.ht + (val * DK + 32 * wv + 4 * q4) * a.dvp + col0 : nullptr;
    float* pw = BACK ? a.w + (val * kC + 4 * q4) * a.dvp + col0 : nullptr;
    auto load_k = [&](const char* at, int s, int to) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int p = 0; p < P; ++p) kf[ii][to][p] = load_frag(at + ((p * 4 + deal.tile(ii)) * KS + s) * kFrag, lane);
    };
    auto load_b = [&](int c) {
        if constexpr (kHold)
#pragma unroll
            for (int s = 0; s < KS; ++s) load_k(pk, s, s);
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            ca[ii] = *reinterpret_cast<const f32x4*>(pca + 16 * deal.tile(ii) + 4 * q4);
#pragma unroll
            for (int x = 0; x < NX; ++x)
                request_forward(
                    seq.n, c, [&](int rows) { v[ii][x].places(a.v.row, rows); }, [&](int at) { v[ii][x].load(at); });
        }
    };
    auto load_c = [&] {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
            ce[ii] = *reinterpret_cast<const f32x4*>(pcb + kC + 16 * i + 4 * q4);
            cb[ii] = *reinterpret_cast<const f32x4*>(pcb + 2 * kC + 16 * i + 4 * q4);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < S; ++p)
                    tm[ii][s][p] = load_frag(pm + (low_frag(i, min(s, i / 2)) * S + p) * kFrag, lane);
        }
    };
    auto load_d = [&] {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < P; ++p) kt[t][s][p] = load_frag(pt + ((p * NT + t) * 2 + s) * kFrag, lane);
        end = co[kC - 1];
    };
#pragma unroll
    for (int ii = 0; ii < NI; ++ii)
#pragma unroll
        for (int x = 0; x < NX; ++x)
            v[ii][x].begin(a.v, seq.row0, hv * a.v.head, 16 * deal.tile(ii) + 4 * q4, col0 + 16 * deal.block(x), a.dv);
    wait_vmem_all();                                 // for H, so that the loop's first wait is not for its operands too
    if (chunks > 0) {
        load_b(0);
        load_c();
        load_d();
    }
    if constexpr (OUT == kOutSame) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) out.tile[ii] = deal.tile(ii);
        out.begin(a, key, val, lane);
        if (chunks > 0) {
            out.load_q(lane);
            out.load_y(lane);
        }
    }
    for (int c = 0; c < chunks; ++c) {
        const bool more = c + 1 < chunks;
        const int rows = more ? kC : tail;
        const char* pk_now = pk;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                put4<S>(hh + place4(cc * KS, 32 * wv + 16 * t + 4 * q4, n), kPh, h[t][cc]);
                if constexpr (BACK)                  // the state before the chunk, for the gradients
#pragma unroll
                    for (int r = 0; r < 4; ++r) ph[(16 * t + r) * a.dvp + 16 * cc] = h[t][cc][r];
            }
        lds_barrier();
        // F = V - a K H
        f32x4 f[NI][NX];
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) f[ii][x] = f32x4{0, 0, 0, 0};
        if constexpr (OUT == kOutSame) out.clear();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if constexpr (!kHold) {
                load_k(pk_now, s, 0);
                if constexpr (OUT == kOutSame) out.load_step(s, 0, lane);
            }
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                bf16x8 hb[S];
                get8<S>(hh + (deal.block(x) * KS + s) * kStep + lane * 8, kPh, hb);
#pragma unroll
                for (int ii = 0; ii < NI; ++ii) f[ii][x] = mma<P, S>(kf[ii][kHold ? s : 0], hb, f[ii][x]);
                if constexpr (OUT == kOutSame) out.add(s, x, hb);
            }
        }
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                f[ii][x] = v[ii][x].get(rows) - ca[ii] * f[ii][x];
                put4<S>(rr + place4(2 * deal.block(x), 16 * deal.tile(ii) + 4 * q4, n), kPl, cb[ii] * f[ii][x]);
            }
        pk += more ? key_step : 0;
        pca += more ? co_step : 0;
        load_b(after(seq.n, c));
        if constexpr (OUT == kOutSame) {
            out.pq += more ? key_step : 0;
            out.load_q(lane);
        }
        lds_barrier();
        // W = F - M R, U = beta W
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int cc = deal.block(x);
                f32x4 m = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s > i / 2) continue;
                    bf16x8 r[S];
                    get8<S>(rr + (2 * cc + s) * kStep + lane * 8, kPl, r);
                    m = mma<S, S>(tm[ii][s], r, m);
                }
                const f32x4 w = f[ii][x] - m, u = cb[ii] * w;
                put4<S>(ue + place4(2 * cc, 16 * i + 4 * q4, n), kPl, ce[ii] * u);
                if constexpr (BACK) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) pw[(16 * i + r) * a.dvp + 16 * cc] = w[r];
                } else {
                    put4<R>(uu + place4(2 * cc, 16 * i + 4 * q4, n), kPl, u);
                }
            }
        }
        pm += more ? m_step : 0;
        pcb += more ? co_step : 0;
        load_c();
        lds_barrier();
        // H'
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            bf16x8 u[2][S];
#pragma unroll
            for (int s = 0; s < 2; ++s) get8<S>(ue + (2 * cc + s) * kStep + lane * 8, kPl, u[s]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                h[t][cc] = end * h[t][cc];
#pragma unroll
                for (int s = 0; s < 2; ++s) h[t][cc] = mma<P, S>(kt[t][s], u[s], h[t][cc]);
            }
        }
        pt += more ? key_step : 0;
        co += more ? co_step : 0;
        load_d();
        if constexpr (OUT == kOutSame) {
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int cc = deal.block(x);
                out.finish(x, uu + 2 * cc * kStep, kPl, po + 16 * cc * E, rows, col0 + 16 * cc < a.dv, lane);
            }
            po += o_step;
            out.py += more ? y_step : 0;
            out.pc += more ? co_step : 0;
            out.load_y(lane);
        }
        if constexpr (BACK) {
            ph += (size_t)a.Hv * DK * a.dvp;
            pw += (size_t)a.Hv * kC * a.dvp;
        }
    }
    if (!BACK && a.S_out) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 32 * wv + 16 * t + 4 * q4 + r, j = col0 + 16 * cc;
                    if (i < a.dk && j < a.dv) a.S_out[state + (size_t)j * a.dk + i] = h[t][cc][r];
                }
    }
}

// ------------------------------------------------------------------ scan, wide
//
// The scan for many slices: a workgroup of four waves takes 64 value columns of a head, and a wave 16
// of them with all of H (d_k rows), so that nothing of a chunk passes between waves: accumulators
// become operands by swaps of lanes.  What the waves share are the chunk's operands, which come to
// LDS once for all four, past the registers.  Each of the three parts of a chunk (K and Q; M;
// K^T and Y) has its place there; the next chunk's part is sent for when every wave is done with it, and
// waited for where two parts of work have passed since.  bf16 rows only: three terms of every
// operand would not fit.  Outputs are formed transposed, so that a lane has four columns of a row.
//
// 81 KB of LDS: two workgroups to a compute unit.  24 prompts, 25331 rows, 32 heads: 443 us, in which
// matrix instructions take a third of the cycles; between them stand the terms of H and the waits
// at the chunk's three barriers.  (rule_scan with two column blocks and the outputs by the state's
// waves: 500 us.  K and Q through prepared operands: 418 us, and rule_prepare 226 in place of 181.)
constexpr int kWide = 64;

// 16 bytes a lane from memory to LDS.  from and to are the wave's; at: the lane's place from there.
__device__ __forceinline__ void send16(const char* from, uint32_t to, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(at), "s"(from) : "memory");
}
template <class X>
__device__ __forceinline__ uint32_t lds_at(X& x) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) X*)&x;
}
// Fragments to LDS, dealt to the waves; `to` and `from` the same for the workgroup.  A wave past the
// last fragment sends that one again, to the same place.
template <int N>
__device__ __forceinline__ void send(const char* from, uint32_t to, int wv, int lane) {
#pragma unroll
    for (int x = 0; x < (N + 3) / 4; ++x) {
        const int f = N % 4 ? min(wv + 4 * x, N - 1) : wv + 4 * x;
        send16(from + f * kFrag, to + f * kFrag, lane * 16);
    }
}

// Tiles 2 s and 2 s + 1 of a column of accumulators, as the terms of one contraction step.
template <int T>
__device__ __forceinline__ void operand(f32x4 x, f32x4 y, bf16x8 (&to)[T]) {
    s16x4 a[T], b[T];
    split4p(x, a);
    split4p(y, b);
#pragma unroll
    for (int p = 0; p < T; ++p) to[p] = stack_pair(a[p], b[p]);
}

template <int DK>
__global__ void __launch_bounds__(256, 2) rule_scan_wide(const RuleArgs a) {
    constexpr int IO = GDN_BF16, KS = DK / 32, NT = DK / 16, S = kSum, R = kRound<IO>;
    constexpr int nK = 4 * KS, nM = kTriFrags * S, nT = 2 * NT, nY = kTriFrags * R;
    __shared__ __attribute__((aligned(16))) char sk[nK * kFrag], sq[nK * kFrag], sm[nM * kFrag], st[nT * kFrag],
        sy[nY * kFrag];
    __shared__ __attribute__((aligned(16))) float sc[2][3 * kC];

    int b, hv, sl;
    scan_place<IO, DK>(a, (a.dvp + kWide - 1) / kWide, b, hv, sl);
    const int hk = hv / a.group;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const RuleSeq seq = rule_seq(a, b);
    const int chunks = chunks_of(seq.n), base = slot_base(seq.row0, b);
    const int tail = last_rows(seq.n);
    const int block = sl * kWide + 16 * wv, col = block + n; // the wave's columns; this lane's
    const bool work = block < a.dvp;                 // columns past d_v have zeros to work on, past dvp no place
    const size_t key = ((size_t)base * a.Hk + hk) * nK * kFrag, val = (size_t)base * a.Hv + hv;
    const size_t key_step = (size_t)a.Hk * nK * kFrag, m_step = (size_t)a.Hv * nM * kFrag, y_step = (size_t)a.Hv * nY * kFrag;
    const size_t co_step = (size_t)a.Hv * 3 * kC;

    f32x4 h[NT];                                     // rows 16 t + 4 q4 + r
    const size_t state = ((size_t)b * a.Hv + hv) * a.dv * a.dk + (size_t)min(col, a.dv - 1) * a.dk;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * t + 4 * q4 + r;
            h[t][r] = a.S0 && i < a.dk && col < a.dv ? a.S0[state + i] : 0.f;
        }
    const char *pt = a.kt + key, *pm = a.tm + val * nM * kFrag, *py = a.ym + val * nY * kFrag;
    const float* pc = a.coef + val * 3 * kC;
    uint16_t v[4][4];                                // of the next chunk: rows 16 i + 4 q4 + r
    const uint16_t* pv = reinterpret_cast<const uint16_t*>(a.v.p) + (seq.row0 + 4 * q4) * a.v.row + hv * a.v.head + min(col, a.dv - 1);
    uint16_t* po = reinterpret_cast<uint16_t*>(a.o.p) + (seq.row0 + n) * a.o.row + hv * a.o.head + block + 4 * q4;
    // the coefficients of chunk c: every lane of the first wave's three quarters sends 16 bytes
    auto send_coef = [&](int c) {
        if (wv == 0 && lane < 3 * kC / 4) send16((const char*)pc, lds_at(sc) + (c & 1) * sizeof(sc[0]), lane * 16);
    };
    // K and Q, as prepared or from the rows themselves: a lane's 16 bytes are eight elements of a row either
    // way.  Rows past the sequence's end are its last row; their coefficients are 0, their outputs not stored.
    const int direct = a.direct;
    auto key_rows = [&](const Rows& x, const char* prepared) {
        return direct ? x.p + (seq.row0 * x.row + hk * x.head) * 2 : prepared + key;
    };
    const char *pk = key_rows(a.k, a.kf), *pq = key_rows(a.q, a.qf);
    auto send_rows = [&](const Rows& x, const char* from, uint32_t to, int rows) {
        const uint32_t row = (uint32_t)x.row * 2;
        const bool part = direct && rows < kC;
#pragma unroll
        for (int y = 0; y < nK / 4; ++y) {
            const int f = wv + 4 * y, i = f / KS, s = f % KS;
            if (part)
                send16(from + 64 * s, to + f * kFrag, min(16 * i + n, rows - 1) * row + 16 * q4);
            else if (direct)
                send16(from + 16 * i * (size_t)row + 64 * s, to + f * kFrag, n * row + 16 * q4);
            else
                send16(from + f * kFrag, to + f * kFrag, lane * 16);
        }
    };
    auto send_k = [&](int rows) {
        send_rows(a.k, pk, lds_at(sk), rows);
        send_rows(a.q, pq, lds_at(sq), rows);
    };
    auto send_t = [&] {
        send<nT>(pt, lds_at(st), wv, lane);
        send<nY>(py, lds_at(sy), wv, lane);
    };
    auto load_v = [&](int rows) {
        if (rows == kC) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[i][r] = pv[(16 * i + r) * a.v.row];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[i][r] = pv[(min(16 * i + 4 * q4 + r, rows - 1) - 4 * q4) * a.v.row];
        }
    };
    if (chunks > 0) {
        send_k(chunks > 1 ? kC : tail);
        send_coef(0);
        load_v(chunks > 1 ? kC : tail);
        send<nM>(pm, lds_at(sm), wv, lane);
    }
    wait_vmem_all();
    for (int c = 0; c < chunks; ++c) {
        const bool more = c + 1 < chunks;
        const int rows = more ? kC : tail;
        const float* co = sc[c & 1];
        lds_barrier();                               // K, Q and M are here, K^T and Y free
        send_t();
        f32x4 f[4], o[4];
        bf16x8 rb[2][S];
        if (work) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = o[i] = f32x4{0, 0, 0, 0};
            bf16x8 k[4][1], q[4][1];
            auto read = [&](const char* from, int s, bf16x8 (&x)[4][1]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i][0] = load_frag(from + (i * KS + s) * kFrag, lane);
            };
            read(sk, 0, k);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                read(sq, s, q);
                hold();
                bf16x8 hb[S];
                operand(h[2 * s], h[2 * s + 1], hb);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = mma<1, S>(k[i], hb, f[i]);
                hold();
                if (s + 1 < KS) read(sk, s + 1, k);
                hold();
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = mma<R, 1>(hb, q[i], o[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 ca = *reinterpret_cast<const f32x4*>(co + 16 * i + 4 * q4);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    f[i][r] = (16 * i + 4 * q4 + r < rows && col < a.dv ? bf16_bits_to_f32(v[i][r]) : 0.f) - ca[r] * f[i][r];
                o[i] = co[16 * i + n] * o[i];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 b0 = *reinterpret_cast<const f32x4*>(co + 2 * kC + 32 * s + 4 * q4);
                const f32x4 b1 = *reinterpret_cast<const f32x4*>(co + 2 * kC + 32 * s + 16 + 4 * q4);
                operand(b0 * f[2 * s], b1 * f[2 * s + 1], rb[s]);
            }
        }
        wait_vmem_all();                             // K^T and Y
        lds_barrier();                               // K and Q are free
        pk += !more ? 0 : direct ? kC * 2 * a.k.row : key_step;
        pq += !more ? 0 : direct ? kC * 2 * a.q.row : key_step;
        pc += more ? co_step : 0;
        send_k(c + 2 < chunks ? kC : tail);
        send_coef(c + 1);
        pv += more ? kC * a.v.row : 0;
        load_v(c + 2 < chunks ? kC : tail);
        bf16x8 ub[2][S], uy[2][R];
        if (work) {
            f32x4 u[4];
            bf16x8 x[2][2][S];
            auto read = [&](int i) {
#pragma unroll
                for (int s = 0; s <= i / 2; ++s)
#pragma unroll
                    for (int p = 0; p < S; ++p) x[i & 1][s][p] = load_frag(sm + (low_frag(i, s) * S + p) * kFrag, lane);
            };
            read(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < 3) read(i + 1);
                hold();
                f32x4 m = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s <= i / 2; ++s) m = mma<S, S>(x[i & 1][s], rb[s], m);
                const f32x4 w = f[i] - m;
                u[i] = *reinterpret_cast<const f32x4*>(co + 2 * kC + 16 * i + 4 * q4) * w;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 e0 = *reinterpret_cast<const f32x4*>(co + kC + 32 * s + 4 * q4);
                const f32x4 e1 = *reinterpret_cast<const f32x4*>(co + kC + 32 * s + 16 + 4 * q4);
                operand(e0 * u[2 * s], e1 * u[2 * s + 1], ub[s]);
                operand(u[2 * s], u[2 * s + 1], uy[s]);
            }
        }
        lds_barrier();                               // M is free
        pm += more ? m_step : 0;
        send<nM>(pm, lds_at(sm), wv, lane);
        if (work) {
            const float end = co[kC - 1];
            bf16x8 k[2][2][2][1];                    // of two tiles, and of the next two
            auto read = [&](int t) {
#pragma unroll
                for (int x = 0; x < 4; ++x) k[t / 2 & 1][x / 2][x % 2][0] = load_frag(st + (2 * t + x) * kFrag, lane);
            };
            bf16x8 y[2][2][R];
            auto read_y = [&](int i) {
#pragma unroll
                for (int s = 0; s <= i / 2; ++s)
#pragma unroll
                    for (int p = 0; p < R; ++p) y[i & 1][s][p] = load_frag(sy + (low_frag(i, s) * R + p) * kFrag, lane);
            };
            read(0);
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                if (t + 2 < NT) read(t + 2);
                else read_y(0);
                hold();
#pragma unroll
                for (int x = 0; x < 2; ++x) h[t + x] = end * h[t + x];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int x = 0; x < 2; ++x) h[t + x] = mma<1, S>(k[t / 2 & 1][x][s], ub[s], h[t + x]);
            }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < 3) read_y(i + 1);
                    hold();
#pragma unroll
                    for (int s = 0; s <= i / 2; ++s) o[i] = mma<R, R>(uy[s], y[i & 1][s], o[i]);
                }
        }
        pt += more ? key_step : 0;
        py += more ? y_step : 0;
        wait_vmem_all();                             // K, Q, M, V and the coefficients
        if (work) {
            // o[i]: row 16 i + n, columns block + 4 q4 + r
            if (a.vo && rows == kC && block + 16 <= a.dv) {
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<s16x4*>(po + 16 * i * a.o.row) = to_bf16x4(o[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * i + n < rows && block + 4 * q4 + r < a.dv) po[16 * i * a.o.row + r] = bf16_rne(o[i][r]);
            }
        }
        po += kC * a.o.row;
    }
    if (a.S_out && col < a.dv)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * t + 4 * q4 + r;
                if (i < a.dk) a.S_out[state + i] = h[t][r];
            }
}

// ------------------------------------------------------------------ scan_back

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row_sum(float x) {
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, false));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x124, 0xf, 0xf, false));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x122, 0xf, 0xf, false));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x121, 0xf, 0xf, false));
    return x;
}

// Tile `second` of the pair of 16 x 16 blocks that stack_pair made one operand of, as accumulators lie.
template <int P>
__device__ __forceinline__ f32x4 rows_of_pair(const bf16x8 (&m)[P], int second) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const u32x4 r = __builtin_bit_cast(u32x4, m[p]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto w = __builtin_amdgcn_permlane16_swap(r[h], r[2 + h], false, false);
            const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
            const uint32_t y = second ? x[1] : x[0];
            v[2 * h] += __uint_as_float(y << 16);
            v[2 * h + 1] += __uint_as_float(y & 0xffff0000u);
        }
    }
    return v;
}

// Sums of the lanes up to each within a row of 16.
__device__ __forceinline__ float row_scan(float x) {
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x111, 0xf, 0xf, true));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x112, 0xf, 0xf, true));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x114, 0xf, 0xf, true));
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x118, 0xf, 0xf, true));
    return x;
}

// rule_scan's shape from the last chunk to the first, the accumulators holding the slice of dH.
// It leaves dH' and dR of every chunk for rule_join, writes dV, and leaves the slice's parts of
// dbeta and of the terms of d ln g that reach the chunk's end: e^(Gamma_C - Gamma_j) k_j . dH' u_j
// of every row, and a_C <H, dH'>.  4 sequences, 6727 rows, 32 heads of 128, bf16: 301 us for 600 MB
// read and 390 written (3.3 TB/s); the longest sequence's 32 chunks are 9.4 us each.
template <int IO, int DK, int NC>
__global__ void __launch_bounds__(DK * 2, IO == GDN_BF16 && DK >= 128 ? 2 : 1) rule_scan_back(const RuleArgs a) {
    constexpr int P = kPlanes<IO>, KS = DK / 32, NW = KS, NT = DK / 16;
    constexpr int S = kSum;
    typedef Deal<NW, NC> D;
    constexpr int NI = D::NI, NX = D::NX;
    constexpr bool kHold = DK * P <= 256;
    constexpr int KH = kHold ? KS : 1;
    constexpr int kPl = NC * 2 * kStep, kPh = NC * KS * kStep; // elements of a term of a tile
    __shared__ __attribute__((aligned(16))) uint16_t hh[S * kPh], od[P * kPl], oa[S * kPl], ou[S * kPl], oz[S * kPl];

    int b, hv, sl;
    const int slices = a.dvp / (16 * NC);
    scan_place<IO, DK>(a, slices, b, hv, sl);
    const int hk = hv / a.group;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const D deal{wv};
    const RuleSeq seq = rule_seq(a, b);
    const int chunks = chunks_of(seq.n), base = slot_base(seq.row0, b);
    const int col0 = sl * 16 * NC + n;
    constexpr size_t kTile = (size_t)P * 4 * KS * kFrag;
    constexpr size_t kTri = (size_t)kTriFrags * kFrag;

    f32x4 dh[2][NC];
    const size_t state = ((size_t)b * a.Hv + hv) * a.dv * a.dk;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 32 * wv + 16 * t + 4 * q4 + r, j = col0 + 16 * c;
                dh[t][c][r] = a.dS_out && i < a.dk && j < a.dv ? a.dS_out[state + (size_t)j * a.dk + i] : 0.f;
            }

    // requested for the chunk before as soon as they have been used, as in rule_scan
    bf16x8 kf[NI][KH][P], kt[2][2][P], qt[2][2][P], tt[NI][2][S], yt[NI][2][S];
    f32x4 ca[NI], ce[NI], cb[NI], w[NI][NX], h[2][NC];
    Rows4<IO> raw[NI][NX];
    float end;
    auto key_of = [&](int c) { return ((size_t)(base + c) * a.Hk + hk) * kTile; };
    auto val_of = [&](int c) { return (size_t)(base + c) * a.Hv + hv; };
    auto load_k = [&](int c, int s, int to) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int p = 0; p < P; ++p)
                kf[ii][to][p] = load_frag(a.kf + key_of(c) + ((p * 4 + deal.tile(ii)) * KS + s) * kFrag, lane);
    };
    auto load_a = [&](int c) {
        const float* from = a.ht + (val_of(c) * DK + 32 * wv + 4 * q4) * a.dvp + col0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                for (int r = 0; r < 4; ++r) h[t][cc][r] = from[(size_t)(16 * t + r) * a.dvp + 16 * cc];
        end = a.coef[val_of(c) * 3 * kC + kC - 1];
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) raw[ii][x].load(c);
    };
    auto load_b = [&](int c) {
        const size_t val = val_of(c);
        if constexpr (kHold)
#pragma unroll
            for (int s = 0; s < KS; ++s) load_k(c, s, s);
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < S; ++p)
                    yt[ii][s][p] = load_frag(a.yt + val * S * kTri + (up_frag(i, max(s, i / 2)) * S + p) * kFrag, lane);
        }
    };
    auto load_c = [&](int c) {
        const size_t val = val_of(c);
        const float* co = a.coef + val * 3 * kC;
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
            ca[ii] = *reinterpret_cast<const f32x4*>(co + 16 * i + 4 * q4);
            ce[ii] = *reinterpret_cast<const f32x4*>(co + kC + 16 * i + 4 * q4);
            cb[ii] = *reinterpret_cast<const f32x4*>(co + 2 * kC + 16 * i + 4 * q4);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < S; ++p)
                    tt[ii][s][p] = load_frag(a.tt + val * S * kTri + (up_frag(i, max(s, i / 2)) * S + p) * kFrag, lane);
            const float* from = a.w + (val * kC + 16 * i + 4 * q4) * a.dvp + col0;
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) w[ii][x][r] = from[(size_t)r * a.dvp + 16 * deal.block(x)];
        }
    };
    auto load_d = [&](int c) {
        const size_t key = key_of(c);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    kt[t][s][p] = load_frag(a.kt + key + ((p * NT + 2 * wv + t) * 2 + s) * kFrag, lane);
                    qt[t][s][p] = load_frag(a.qt + key + ((p * NT + 2 * wv + t) * 2 + s) * kFrag, lane);
                }
    };
    auto places = [&](int rows) {
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) raw[ii][x].places(a.d_o.row, rows);
    };
#pragma unroll
    for (int ii = 0; ii < NI; ++ii)
#pragma unroll
        for (int x = 0; x < NX; ++x)
            raw[ii][x].begin(a.d_o, seq.row0, hv * a.d_o.head, 16 * deal.tile(ii) + 4 * q4, col0 + 16 * deal.block(x), a.dv);
    wait_vmem_all();
    if (chunks > 0) {
        request_back_first(seq.n, places, load_a);
        load_b(chunks - 1);
        load_c(chunks - 1);
        load_d(chunks - 1);
    }
    for (int c = chunks - 1; c >= 0; --c) {
        const size_t val = val_of(c);
        const int next = before(c);
        // dH' and dO to LDS, and a_C <H, dH'>
        f32x4 d_o[NI][NX];
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int i = deal.tile(ii), cc = deal.block(x);
                d_o[ii][x] = raw[ii][x].get(seq.n - c * kC);
                put4<P>(od + place4(2 * cc, 16 * i + 4 * q4, n), kPl, d_o[ii][x]);
            }
        float pa = 0.f;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                put4<S>(hh + place4(cc * KS, 32 * wv + 16 * t + 4 * q4, n), kPh, dh[t][cc]);
                float* to = a.dht + (val * DK + 32 * wv + 16 * t + 4 * q4) * a.dvp + col0 + 16 * cc;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    to[(size_t)r * a.dvp] = dh[t][cc][r];
                    pa += h[t][cc][r] * dh[t][cc][r];
                }
            }
        const float decay = end;
        pa = row_sum(decay * pa);
        if (n == 0) a.pa[((val * slices + sl) * NW + wv) * 4 + q4] = pa;
        load_a(next);
        lds_barrier();
        // dU = e^(Gamma_C - Gamma) K dH' + Y^T dO
        f32x4 du[NI][NX], pe[NI];
#pragma unroll
        for (int ii = 0; ii < NI; ++ii)
#pragma unroll
            for (int x = 0; x < NX; ++x) du[ii][x] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if constexpr (!kHold) load_k(c, s, 0);
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                bf16x8 hb[S];
                get8<S>(hh + (deal.block(x) * KS + s) * kStep + lane * 8, kPh, hb);
#pragma unroll
                for (int ii = 0; ii < NI; ++ii) du[ii][x] = mma<P, S>(kf[ii][kHold ? s : 0], hb, du[ii][x]);
            }
        }
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
            pe[ii] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int cc = deal.block(x);
                f32x4 s = ce[ii] * du[ii][x];
                pe[ii] += s * cb[ii] * w[ii][x];
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    if (st < i / 2) continue;
                    bf16x8 d[P];
                    get8<P>(od + (2 * cc + st) * kStep + lane * 8, kPl, d);
                    s = mma<S, P>(yt[ii][st], d, s);
                }
                du[ii][x] = s;
                put4<S>(ou + place4(2 * cc, 16 * i + 4 * q4, n), kPl, cb[ii] * s);
                put4<S>(oa + place4(2 * cc, 16 * i + 4 * q4, n), kPl, ca[ii] * d_o[ii][x]);
            }
        }
        load_b(next);
        lds_barrier();
        // dR = dU - M^T beta dU
#pragma unroll
        for (int ii = 0; ii < NI; ++ii) {
            const int i = deal.tile(ii);
            f32x4 pb = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int cc = deal.block(x);
                f32x4 m = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s < i / 2) continue;
                    bf16x8 u[S];
                    get8<S>(ou + (2 * cc + s) * kStep + lane * 8, kPl, u);
                    m = mma<S, S>(tt[ii][s], u, m);
                }
                const f32x4 dr = du[ii][x] - m, dv = cb[ii] * dr;
                put4<S>(oz + place4(2 * cc, 16 * i + 4 * q4, n), kPl, -ca[ii] * dv);
                float* to = a.dr + (val * kC + 16 * i + 4 * q4) * a.dvp + col0 + 16 * cc;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = c * kC + 16 * i + 4 * q4 + r, col = col0 + 16 * cc;
                    to[(size_t)r * a.dvp] = dr[r];
                    if (row < seq.n && col < a.dv)
                        put_io<IO>(a.dv_out.p, (seq.row0 + row) * a.dv_out.row + hv * a.dv_out.head + col, dv[r]);
                }
                pb += dr * w[ii][x];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) pb[r] = row_sum(pb[r]), pe[ii][r] = row_sum(pe[ii][r]);
            if (n == 0) {
                // with eight waves a slice's two column blocks are two parts
                const size_t at = ((val * slices + sl) * (NC / NX) + (NX < NC ? deal.block(0) : 0)) * kC + 16 * i + 4 * q4;
                *reinterpret_cast<f32x4*>(a.pb + at) = pb;
                *reinterpret_cast<f32x4*>(a.pe + at) = pe[ii];
            }
        }
        load_c(next);
        lds_barrier();
        // dH
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            bf16x8 u[2][S], z[2][S];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                get8<S>(oa + (2 * cc + s) * kStep + lane * 8, kPl, u[s]);
                get8<S>(oz + (2 * cc + s) * kStep + lane * 8, kPl, z[s]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                dh[t][cc] = decay * dh[t][cc];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    dh[t][cc] = mma<P, S>(qt[t][s], u[s], dh[t][cc]);
                    dh[t][cc] = mma<P, S>(kt[t][s], z[s], dh[t][cc]);
                }
            }
        }
        load_d(next);
    }
    if (a.dS0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 32 * wv + 16 * t + 4 * q4 + r, j = col0 + 16 * cc;
                    if (i < a.dk && j < a.dv) a.dS0[state + (size_t)j * a.dk + i] = dh[t][cc][r];
                }
    }
}

// ------------------------------------------------------------------ join
//
// dQ, dK and what the gates' gradients need, one workgroup per (chunk slot, key head) and d_k / 16
// waves: wave w owns columns 16 w .. 16 w + 15 of dQ and dK and sums them over the key head's value
// heads in registers, so that gradients of shared heads need no atomics.  The 16 x 16 tiles of
// dO U^T and dR U^T below the diagonal are dealt to the waves; value columns go by blocks of 64, and
// a block's rows are requested while the block before it is worked on.
//
// d ln g_t (rule_gates) is the sum of what every path across row t carries, a path from row j or from
// the chunk's start to row i or to the chunk's end:
//
//     sum_(i >= t > j) Z_ij + sum_(i >= t) h_i + sum_(j < t) e_j + a_C <H, dH'>,
//     Z = P o Q K^T + G o K K^T,  h_i = a_i (dO_i . H^T q_i - beta_i dR_i . H^T k_i)
//
// A running sum of differences over the rows (v . dv - o . do) would be shorter, but its terms do
// not shrink with the gate: a head that forgets at once would get its small gradient as a
// difference of large ones.
//
// 6727 rows, 32 heads of 128, bf16: 290 us for 790 MB read (H and dH' in fp32, the most of it), 2.7
// TB/s.  129 KB of LDS leave one workgroup to a unit, whose waves wait for half of their time.
template <int IO, int DK>
__global__ void __launch_bounds__(DK * 4) rule_join(const RuleArgs a) {
    constexpr int P = kPlanes<IO>, KS = DK / 32, NT = DK / 16, NW = NT, VB = 64, LD = VB + 8;
    constexpr int S = kSum, R = kRound<IO>, D = R;  // D: terms of dH', P^T and G in dK
    constexpr int kPl = kC * LD, kSq = kC * kTp;
    constexpr int ND = (10 + NW - 1) / NW;           // tiles below or on the diagonal, per wave
    constexpr size_t kTile = (size_t)P * 4 * KS * kFrag;
    // value rows of a block and, with bf16, of the next; the 64 x 64 matrices in the first one's place
    constexpr int NB = IO == GDN_BF16 ? 2 : 1, kBlk = (2 * S + P) * kPl;
    __shared__ __attribute__((aligned(16))) uint16_t lds[NB * kBlk];
    static_assert(kBlk >= (S + 2 * D) * kSq, "the matrices fit");
    __shared__ double gam[kC];
    __shared__ __attribute__((aligned(16))) float coef[3][kC];
    uint16_t *sp = lds, *spt = lds + S * kSq, *sg = spt + D * kSq;

    const int slot = blockIdx.x, hk = blockIdx.y;
    const RuleChunk ch = rule_chunk(a, slot);
    if (ch.n == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q4 = lane >> 4;
    const size_t key = ((size_t)slot * a.Hk + hk) * kTile;
    const int col = 16 * wv + n;

    f32x4 dq[4], dk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[i] = dk[i] = f32x4{0, 0, 0, 0};
    auto tile_row = [](int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; };
    auto tile_col = [&](int t) { return t - tile_row(t) * (tile_row(t) + 1) / 2; };
    // rows of U (as W), dR and dO of one block: 8 columns of a row to a thread
    constexpr int kPiecesAll = kC * VB / 8, kPieces = (kPiecesAll + NW * 64 - 1) / (NW * 64);
    f32x4 bw[kPieces][2], by[kPieces][2];
    float bb[kPieces];
    Planes<IO> bo[kPieces];
    auto load_block = [&](int hv, int v0) {
        const size_t val = (size_t)slot * a.Hv + hv;
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            const int p = min(tid + x * NW * 64, kPiecesAll - 1), r = p / (VB / 8), c = min(v0 + p % (VB / 8) * 8, a.dvp - 8);
            const size_t at = (val * kC + r) * a.dvp + c;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bw[x][j] = *reinterpret_cast<const f32x4*>(a.w + at + 4 * j);
                by[x][j] = *reinterpret_cast<const f32x4*>(a.dr + at + 4 * j);
            }
            bb[x] = a.coef[(val * 3 + 2) * kC + r];
            const bool live = r < ch.n;
            bo[x] = load_row8<IO>(a.d_o.p, (ch.row0 + (live ? r : 0)) * a.d_o.row + (int64_t)hv * a.d_o.head, c, a.dv,
                                  a.vdo, live);
        }
    };
    load_block(hk * a.group, 0);
    for (int gi = 0; gi < a.group; ++gi) {
        const int hv = hk * a.group + gi;
        const size_t val = (size_t)slot * a.Hv + hv;
        f32x4 dy[ND], dx[ND], aq[4], t1[4], t2[4];
#pragma unroll
        for (int i = 0; i < ND; ++i) dy[i] = dx[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) aq[i] = t1[i] = t2[i] = f32x4{0, 0, 0, 0};

        // this lane's row of H and dH': 8 value columns of a contraction step
        const float* ph = a.ht + (val * DK + col) * a.dvp + 8 * q4;
        const float* pd = a.dht + (val * DK + col) * a.dvp + 8 * q4;
        f32x4 hx[2], dx2[2];
        auto load_h = [&](int v) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                hx[j] = *reinterpret_cast<const f32x4*>(ph + v + 4 * j);
                dx2[j] = *reinterpret_cast<const f32x4*>(pd + v + 4 * j);
            }
        };
        load_h(0);
        for (int v0 = 0; v0 < a.dvp; v0 += VB) {
            const int width = min(VB, a.dvp - v0);
            uint16_t* su = lds + (NB == 2 ? v0 / VB % 2 : 0) * kBlk;
            uint16_t *sr = su + S * kPl, *so = sr + S * kPl;
            if (NB == 1 || v0 == 0) __syncthreads();
            if (v0 == 0 && tid < kC) {
                gam[tid] = a.gam[val * kC + tid];
#pragma unroll
                for (int x = 0; x < 3; ++x) coef[x][tid] = a.coef[(val * 3 + x) * kC + tid];
            }
#pragma unroll
            for (int x = 0; x < kPieces; ++x) {
                const int p = tid + x * NW * 64, r = p / (VB / 8), c = p % (VB / 8) * 8;
                if (kPiecesAll % (NW * 64) != 0 && p >= kPiecesAll) break;
                float u[8], d[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = bb[x] * bw[x][j / 4][j % 4], d[j] = by[x][j / 4][j % 4];
                bf16x8 us[S], ds[S];
                split8(u, us);
                split8(d, ds);
#pragma unroll
                for (int t = 0; t < S; ++t) {
                    *reinterpret_cast<bf16x8*>(su + t * kPl + r * LD + c) = us[t];
                    *reinterpret_cast<bf16x8*>(sr + t * kPl + r * LD + c) = ds[t];
                }
#pragma unroll
                for (int t = 0; t < P; ++t) *reinterpret_cast<bf16x8*>(so + t * kPl + r * LD + c) = bo[x].p[t];
            }
            __syncthreads();
            {
                const bool same = v0 + VB < a.dvp;   // the next block, or the last one again
                load_block(same || gi + 1 == a.group ? hv : hv + 1, same ? v0 + VB : 0);
            }
            for (int s = 0; s < width / 32; ++s) {
                const int at = 32 * s + 8 * q4;
                bf16x8 h[S], d[D];
                {
                    float x[8], y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = hx[j / 4][j % 4], y[j] = dx2[j / 4][j % 4];
                    split8(x, h);
                    split8(y, d);
                }
                load_h(min(v0 + 32 * s + 32, a.dvp - 32));
                // dO U^T and dR U^T
#pragma unroll
                for (int x = 0; x < ND; ++x) {
                    const int t = wv + x * NW;
                    if (t >= 10) break;
                    const int i = tile_row(t), j = tile_col(t);
                    bf16x8 u[S], o[P], r[S];
                    get8<S>(su + (16 * j + n) * LD + at, kPl, u);
                    get8<P>(so + (16 * i + n) * LD + at, kPl, o);
                    get8<S>(sr + (16 * i + n) * LD + at, kPl, r);
                    dy[x] = mma<P, S>(o, u, dy[x]);
                    dx[x] = mma<S, S>(r, u, dx[x]);
                }
                // dO H^T, dR H^T and U dH'^T; an operand is read as soon as the one before it is used
                bf16x8 u[R], o[P], r[S];
                const int row = n * LD + at;
                get8<P>(so + row, kPl, o);
                get8<S>(sr + row, kPl, r);
                get8<R>(su + row, kPl, u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int next = row + 16 * (i + 1) * LD;
                    hold();
                    aq[i] = mma<P, S>(o, h, aq[i]);
                    if (i < 3) get8<P>(so + next, kPl, o);
                    hold();
                    t2[i] = mma<S, S>(r, h, t2[i]);
                    if (i < 3) get8<S>(sr + next, kPl, r);
                    hold();
                    t1[i] = mma<R, D>(u, d, t1[i]);
                    if (i < 3) get8<R>(su + next, kPl, u);
                }
            }
        }
        // requested before the barrier: the products that Z takes, and the operands of P and G
        f32x4 kk[ND], qk[ND];
#pragma unroll
        for (int x = 0; x < ND; ++x) {
            const f32x4* gram =
                reinterpret_cast<const f32x4*>(a.gram) + (((size_t)slot * a.Hk + hk) * 10 + min(wv + x * NW, 9)) * 128;
            kk[x] = gram[lane];
            qk[x] = gram[64 + lane];
        }
        bf16x8 kt[2][P], qt[2][P];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                kt[s][p] = load_frag(a.kt + key + ((p * NT + wv) * 2 + s) * kFrag, lane);
                qt[s][p] = load_frag(a.qt + key + ((p * NT + wv) * 2 + s) * kFrag, lane);
            }
        __syncthreads();
        // P, its transpose, G + G^T, and the sums of Z
#pragma unroll
        for (int x = 0; x < ND; ++x) {
            const int t = wv + x * NW;
            if (t >= 10) break;
            const int i = tile_row(t), j = tile_col(t);
            f32x4 p, g;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * q4 + r, c = 16 * j + n;
                const float d = c <= row ? exp2f((float)(gam[row] - gam[c])) : 0.f;
                p[r] = c <= row ? d * dy[x][r] : 0.f;
                g[r] = c < row ? -coef[2][row] * d * dx[x][r] : 0.f;
            }
            // z: the sums of Z's columns up to this one; of column 15, of the whole row.  Row t = 16 j + n + 1
            // is crossed by the rows i >= t of them.
            float cross = 0.f;
            float* zs = a.zs + val * 320 + 16 * t;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 4 * q4 + r;
                const float z = row_scan(i == j && n == row ? 0.f : p[r] * qk[x][r] + g[r] * kk[x][r]);
                if (n == 15) zs[160 + row] = z;
                if (i > j || row > n) cross += z;
            }
            cross += __shfl_xor(cross, 16);
            cross += __shfl_xor(cross, 32);
            if (q4 == 0) zs[n < 15 ? n + 1 : 0] = n < 15 ? cross : 0.f;
            s16x4 ps[S], gs[D];
            split4p(p, ps);
            split4p(g, gs);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * q4 + r, c = 16 * j + n;
#pragma unroll
                for (int y = 0; y < S; ++y) sp[y * kSq + row * kTp + c] = (uint16_t)ps[y][r];
#pragma unroll
                for (int y = 0; y < D; ++y) {        // on the diagonal block the upper half comes from below
                    if (c <= row) sg[y * kSq + row * kTp + c] = (uint16_t)gs[y][r];
                    if (c < row) sg[y * kSq + c * kTp + row] = (uint16_t)gs[y][r];
                }
                if (i == j && (i & 1) == 0) {        // the zero tile that shares an operand with this one
#pragma unroll
                    for (int y = 0; y < S; ++y) sp[y * kSq + row * kTp + c + 16] = 0;
#pragma unroll
                    for (int y = 0; y < D; ++y) spt[y * kSq + (row + 16) * kTp + c] = 0;
                }
            }
            put4<D>(spt + (16 * j + n) * kTp + 16 * i + 4 * q4, kSq, p);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 ca = *reinterpret_cast<const f32x4*>(&coef[0][16 * i + 4 * q4]);
            const f32x4 ce = *reinterpret_cast<const f32x4*>(&coef[1][16 * i + 4 * q4]);
            const f32x4 cb = *reinterpret_cast<const f32x4*>(&coef[2][16 * i + 4 * q4]);
            const f32x4 back = ca * cb * t2[i];
            f32x4 xq = ca * aq[i], xk = ce * t1[i] - back;
            f32x4 h = rows_of_pair(qt[i / 2], i & 1) * xq - rows_of_pair(kt[i / 2], i & 1) * back;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int at = (16 * i + n) * kTp + 32 * s + 8 * q4;
                bf16x8 m[S], g[D];
                if (s <= i / 2) {
                    get8<S>(sp + at, kSq, m);
                    xq = mma<S, P>(m, kt[s], xq);
                }
                if (s >= i / 2) {
                    get8<D>(spt + at, kSq, g);
                    xk = mma<D, P>(g, qt[s], xk);
                }
                get8<D>(sg + at, kSq, g);
                xk = mma<D, P>(g, kt[s], xk);
            }
            dq[i] += xq;
            dk[i] += xk;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = row_sum(h[r]);
            if (n == 0) *reinterpret_cast<f32x4*>(a.hs + (val * NT + wv) * kC + 16 * i + 4 * q4) = h;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * q4 + r;
            if (row < ch.n && col < a.dk) {
                put_io<IO>(a.dq.p, (ch.row0 + row) * a.dq.row + hk * a.dq.head + col, dq[i][r]);
                put_io<IO>(a.dk_out.p, (ch.row0 + row) * a.dk_out.row + hk * a.dk_out.head + col, dk[i][r]);
            }
        }
}

// The gates' gradients of one (chunk slot, value head): a wave, lane t for row t.  parts and waves:
// what a slice's waves left in pb and pe, and in pa; hsums: in hs.
template <int IO>
__global__ void __launch_bounds__(64) rule_gates(const RuleArgs a, int parts, int waves, int hsums) {
    const int slot = blockIdx.x, hv = blockIdx.y, lane = threadIdx.x;
    const RuleChunk ch = rule_chunk(a, slot);
    if (ch.n == 0) return;
    const size_t val = (size_t)slot * a.Hv + hv;
    __shared__ __attribute__((aligned(16))) float z[320];
    float zr[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) zr[i] = a.zs[val * 320 + 64 * i + lane];
    // the lane's column of `count` rows, eight requests at a time
    auto column = [&](const float* rows, int count) {
        double sum = 0;
        for (int w = 0; w < count; w += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = rows[(size_t)min(w + i, count - 1) * kC + lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += w + i < count ? x[i] : 0.f;
        }
        return sum;
    };
    double own = column(a.hs + val * hsums * kC, hsums);
    double to_end = column(a.pe + val * parts * kC, parts);
    const float db = (float)column(a.pb + val * parts * kC, parts);
    double lead = 0;
    for (int s = lane; s < waves * 4; s += 64) lead += a.pa[val * waves * 4 + s];
#pragma unroll
    for (int i = 0; i < 5; ++i) z[64 * i + lane] = zr[i];
    const double mine = to_end;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        const double y = __shfl_down(own, off), x = __shfl_up(to_end, off);
        if (lane + off < 64) own += y;
        if (lane >= off) to_end += x;
        lead += __shfl_xor(lead, off);
    }
    double d = lead + own + to_end - mine;
    __syncthreads();
    const int T = lane / 16, n = lane % 16;
#pragma unroll
    for (int t = 0; t < 10; ++t) {
        const int i = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, j = t - i * (i + 1) / 2;
        if (j == T) d += z[16 * t + n];
        if (i == j) continue;
        const int first = j < T && T <= i ? (T == i ? n : 0) : 16; // rows of this tile that cross row t
#pragma unroll
        for (int r = 0; r < 16; ++r) d += r >= first ? z[160 + 16 * t + r] : 0.f;
    }
    if (lane < ch.n) {
        const int64_t at = (ch.row0 + lane) * a.Hv + hv;
        a.dlog_g[at] = (float)d;
        a.dbeta[at] = db;
    }
}

// ------------------------------------------------------------------ launchers

// Workgroups of a scan with slices of 16 value columns.
inline int64_t slices_of_16(const RuleArgs& a) { return (int64_t)a.B * a.Hv * (a.dvp / 16); }

template <int DK>
hipError_t scan_wide_launch(const RuleArgs& a, hipStream_t stream) {
    return launch(rule_scan_wide<DK>, dim3(a.B * a.Hv * ((a.dvp + kWide - 1) / kWide)), dim3(256), 0, stream, a);
}

template <int IO, int DK, int NC, int OUT>
hipError_t scan_launch(const RuleArgs& a, hipStream_t stream) {
    const int waves = DK / 32 + (OUT == kOutOwn ? kOutWaves<DK> : 0);
    return launch(rule_scan<IO, DK, NC, OUT>, dim3(a.B * a.Hv * (a.dvp / (16 * NC))), dim3(waves * 64), 0, stream, a);
}

// Which scan, by the number of slices of 16 columns (bf16, 32 heads, uneven lengths up to 2048; us with
// what rule_prepare takes before it):
//   d_k 128, slices           512    768   1024   2048   4096
//   outputs by own waves      134    116    209    334    703   narrowest, shortest chunk of all
//   two column blocks         135    123    182    256    499   half the operands read per column
//   wide                      203    189    219    290    442   a quarter, longest chunk of all
//   d_k 64, slices            512   1024   1536   2048   4096
//   outputs by own waves      117    162    361    337    674
//   two column blocks         160    189    327    291    580
//   wide                      166    185    305    290    522
// Waves of their own for the outputs while the workgroups have places (a workgroup of d_k 64 has half
// the waves); half as many again would still be no loss at d_k 128.  The wide one where it has more
// workgroups than places.  Slices alone decide, lengths do not: a sequence of many rows among
// enough short ones takes the wide scan, 5 us a chunk, where the narrow one takes 1.9.
template <int DK>
constexpr int64_t kFewSlices = kPlaces * 128 / DK;
template <int IO, int DK>
hipError_t rule_forward_launch(const RuleArgs& args, hipStream_t stream) {
    RuleArgs a = args;
    hipError_t e = hipSuccess;
    const bool wide = IO == GDN_BF16 && DK <= 128 && slices_of_16(a) > 4 * kPlaces;
    // The wide scan takes keys and queries from their rows where these are whole operands, 16 bytes at a time,
    // and 64 of them within a lane's 32-bit offset (25331 rows, 16 heads of 128: 646 us for
    // both kernels, 670 through prepared operands, which are 210 MB more to write).
    constexpr int64_t kNear = 1 << 24;
    a.direct = wide && a.dk == DK && a.vk && a.vq && a.k.row <= kNear && a.q.row <= kNear;
    if (a.T > 0)
        e = launch(rule_prepare<IO, DK, false>, dim3(a.n_slots, a.Hk), dim3(256), 0, stream, a);
    if (e != hipSuccess) return e;
    if constexpr (DK == 256) {
        return scan_launch<IO, DK, 2, kOutSame>(a, stream);
    } else {
        if (slices_of_16(a) <= kFewSlices<DK>) return scan_launch<IO, DK, 1, kOutOwn>(a, stream);
        if constexpr (IO == GDN_BF16)
            if (wide) return scan_wide_launch<DK>(a, stream);
        return scan_launch<IO, DK, 2, kOutSame>(a, stream);
    }
}

template <int IO, int DK, int NC>
hipError_t back_launch(const RuleArgs& a, hipStream_t stream) {
    constexpr int NW = DK / 32;
    const int slices = a.dvp / (16 * NC);
    hipError_t e = hipSuccess;
    if (a.T > 0) {
        e = launch(rule_prepare<IO, DK, true>, dim3(a.n_slots, a.Hk), dim3(256), 0, stream, a);
        if (e == hipSuccess) e = scan_launch<IO, DK, NC, kOutNone>(a, stream);
    }
    if (e == hipSuccess)
        e = launch(rule_scan_back<IO, DK, NC>, dim3(a.B * a.Hv * slices), dim3(DK * 2), 0, stream, a);
    if (e == hipSuccess && a.T > 0) {
        e = launch(rule_join<IO, DK>, dim3(a.n_slots, a.Hk), dim3(DK * 4), 0, stream, a);
        if (e == hipSuccess)
            e = launch(rule_gates<IO>, dim3(a.n_slots, a.Hv), dim3(64), 0, stream, a, slices * NC / Deal<NW, NC>::NX,
                       slices * NW, DK / 16);
    }
    return e;
}

// One column block to a workgroup while they have places.  Both scans, one block against two, bf16, 32 heads, us:
// d_k 128, 512 slices 289 and 306, 768 slices 398 and 355; d_k 64, 512 slices 249 and 263, 768 slices 353 and 317.
template <int IO, int DK>
hipError_t rule_backward_launch(const RuleArgs& a, hipStream_t stream) {
    if constexpr (DK == 256)
        return back_launch<IO, DK, 2>(a, stream);
    else
        return slices_of_16(a) <= kPlaces ? back_launch<IO, DK, 1>(a, stream) : back_launch<IO, DK, 2>(a, stream);
}

}  // namespace gdn
