// score.hip -- log-probabilities of given tokens, entropy and best alternatives of rows of
// logits, and their gradient; kernels and C ABI.
//
// One pass over a row keeps, per thread, the running maximum m and, with d = (x - m) log2 e, s = sum
// 2^d and t = sum 2^d d; a change of m by d turns them into 2^d s and 2^d (t + d s).  Then lse = m +
// ln s and the entropy is ln s - (t / s) ln 2.  Both kernels are bound by the logits' bytes; the
// exponentials and sums take two thirds of that time.  8192 rows of 65536, bf16: 205 us, 5.2 TB/s read;
// the gradient of 4096 such rows: 195 us, 5.5 TB/s read and written.
//
// The best alternative is in the piece of 16 bytes where its thread last raised its maximum.  More
// alternatives come of a bound that at least k of the threads' maxima reach: the least maximum of
// eight groups of threads, or, past eight, one found by halving that few more than k reach.  Threads
// whose own maximum reaches it read their elements once more; what reaches it is ordered by
// counting.  Where more elements reach it than fit, as in rows that are masked nearly
// everywhere, the k-th best is found byte by byte of (value, index).
#include <float.h>
#include <stdint.h>

#include "attn_common.hpp"
#include "gdn_score.h"
#include "mfma_tiles.hpp"

namespace gdn {
namespace {

constexpr int kMaxTop = 64;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// What stands in for -inf where it would meet a factor of 0.
constexpr float kFar = -1e30f;

struct ScoreArgs {
    int64_t stride;
    int vocab, topk, parts, part;            // part: elements of a part of a row
    const char* logits;
    const int32_t* tokens;
    float* logp;
    float* entropy;
    float* lse;
    float* top_logp;
    int32_t* top_tok;
    float* stat;                             // [rows][parts][3], where rows have parts
    uint64_t* best;                          // [rows][parts][topk]
};

template <int IO>
constexpr int kPer = IO == GDN_BF16 ? 8 : 4; // elements of 16 bytes

template <int IO>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[kPer<IO>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IO == GDN_BF16) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(v[i]);
        }
    }
}

// Elements lo .. hi - 1 of a row: `head` single ones up to a multiple of 16 bytes, `pieces` of 16
// bytes, and single ones to the end.  A thread has the pieces and single ones of its number.
template <int IO>
struct Span {
    const char* row;                         // element 0
    int lo, hi, head, pieces;
    __device__ Span(const char* row_, int lo_, int hi_) : row(row_), lo(lo_), hi(hi_) {
        constexpr int e = IO == GDN_BF16 ? 2 : 4;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (uintptr_t)lo * e;
        head = min(hi - lo, (int)((16 - (at & 15)) & 15) / e);
        pieces = (hi - lo - head) / kPer<IO>;
    }
    __device__ const u32x4* piece(int p) const {
        return reinterpret_cast<const u32x4*>(row + (size_t)(lo + head) * (IO == GDN_BF16 ? 2 : 4)) + p;
    }
    __device__ int first_of(int p) const { return lo + head + p * kPer<IO>; }
    __device__ int tail() const { return first_of(pieces); }
    // f(x, index) for the elements of piece p, v, less all of it below `least` (NaN: none is)
    template <class F>
    __device__ __forceinline__ void elements(u32x4 v, int p, float least, F f) const {
        float x[kPer<IO>];
        unpack<IO>(v, x);
        float most = x[0];
#pragma unroll
        for (int i = 1; i < kPer<IO>; ++i) most = fmaxf(most, x[i]);
        if (most < least) return;
#pragma unroll
        for (int i = 0; i < kPer<IO>; ++i) f(x[i], first_of(p) + i);
    }
    // ... of the single elements of this thread
    template <class F>
    __device__ __forceinline__ void singles(F f) const {
        const int t = threadIdx.x;
        if (t < head) f(ld_io<IO>(row, lo + t), lo + t);
        if (t < hi - tail()) f(ld_io<IO>(row, tail() + t), tail() + t);
    }
    // ... and of all of its elements, read again, four pieces at once
    template <class F>
    __device__ void each(int threads, float least, F f) const {
        singles(f);
        for (int p0 = threadIdx.x; p0 < pieces; p0 += 4 * threads) {
            u32x4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = *piece(min(p0 + u * threads, pieces - 1));
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (p0 + u * threads < pieces) elements(v[u], p0 + u * threads, least, f);
        }
    }
};

struct Stat {
    float m, s, t;
    __device__ void raise(float to) {        // to >= m
        const float d = fmaxf((m - to) * kLog2E, kFar), e = __builtin_amdgcn_exp2f(d);
        t = e * (t + d * s);
        s = e * s;
        m = to;
    }
    __device__ void add(float x) {           // x <= m
        const float d = (x - m) * kLog2E, e = __builtin_amdgcn_exp2f(d);
        s += e;
        t = fmaf(e, fmaxf(d, kFar), t);
    }
    __device__ void join(Stat o) {
        const float to = fmaxf(m, o.m);
        raise(to);
        o.raise(to);
        s += o.s;
        t += o.t;
    }
};
// Floats as unsigned numbers in the same order: -0 is 0, NaN is above all.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0xffffffffu : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0xffffffffu ? __builtin_nanf("") : __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// By value, then by the lower index (24 bits).
__device__ __forceinline__ uint64_t rank_of(float x, int i) {
    return (uint64_t)order_of(x) << 24 | (0xffffffu - (uint32_t)i);
}
__device__ __forceinline__ int index_of(uint64_t r) { return 0xffffff - (int)(r & 0xffffffu); }

// ln p of a logit, and the row's results.
struct Row {
    float m, log_s, mean;
    __device__ explicit Row(const Stat& a) {
        m = a.s == 0.f ? __builtin_nanf("") : a.m; // no finite logit
        log_s = logf(a.s);
        mean = a.t / a.s * kLn2;
    }
    __device__ float logp(float x) const { return (x - m) - log_s; }
};

template <int IO>
__device__ void write_row(const ScoreArgs& a, int64_t row, const Row& r) {
    if (a.lse) a.lse[row] = r.m + r.log_s;
    if (a.entropy) a.entropy[row] = r.m != r.m ? r.m : r.log_s - r.mean;
    if (a.tokens) {
        const int t = a.tokens[row];
        const bool in = t >= 0 && t < a.vocab;
        a.logp[row] = in ? r.logp(ld_io<IO>(a.logits, (size_t)(row * a.stride + t))) : __builtin_nanf("");
    }
}

// The first topk of the n ranks in `c`, in order.  Every rank is different.
template <class F>
__device__ void put_best(const uint64_t* c, int n, int topk, int threads, F put) {
    for (int i = threadIdx.x; i < n; i += threads) {
        const uint64_t mine = c[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += c[j] > mine;
        if (above < topk) put(above, mine);
    }
}

template <int IO, int NT>
__global__ void __launch_bounds__(NT) score_rows(const ScoreArgs a) {
    constexpr int NW = NT / 64, U = 8, kCap = 512;
    __shared__ Stat stats[NW];
    __shared__ uint32_t lows[NW], highs[NW];
    __shared__ int reach[2][NW];
    __shared__ uint64_t cand[kCap];
    __shared__ uint32_t hist[256];
    __shared__ int count;
    __shared__ uint64_t prefix;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const Span<IO> sp(a.logits + (size_t)(row * a.stride) * (IO == GDN_BF16 ? 2 : 4), part * a.part,
                      min(a.vocab, (part + 1) * a.part));
    Stat st{-FLT_MAX, 0.f, 0.f};
    int where = -1;                                  // of the maximum: a piece; or a single element, before or after
    auto single = [&](float x, int at) {
        if (x > st.m) {
            st.raise(x);
            where = at;
        }
        st.add(x);
    };
    if (tid < sp.head) single(ld_io<IO>(sp.row, sp.lo + tid), -1);
    u32x4 v[U];                                      // of a short row, all of this thread's pieces to the end
    for (int p0 = tid; p0 < sp.pieces; p0 += NT * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *sp.piece(min(p0 + u * NT, sp.pieces - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * NT;
            if (p >= sp.pieces) break;
            float x[kPer<IO>];
            unpack<IO>(v[u], x);
            float to = x[0];
#pragma unroll
            for (int i = 1; i < kPer<IO>; ++i) to = fmaxf(to, x[i]);
            if (to > st.m) {
                st.raise(to);
                where = p;
            }
#pragma unroll
            for (int i = 0; i < kPer<IO>; ++i) st.add(x[i]);
        }
    }
    if (tid < sp.hi - sp.tail()) single(ld_io<IO>(sp.row, sp.tail() + tid), -2);
    // a thread that saw NaN (its sum is) has an element above all
    const uint32_t mine = st.s != st.s ? 0xffffffffu : order_of(st.m);
    const int topk = a.topk;
    uint32_t low = mine;                             // of groups: their maximum, then the least of them
    int width = 64;                                  // lanes of a group
    while (topk > 1 && NT / width < topk) width /= 2;
    for (int off = 1; off < width; off *= 2) low = max(low, (uint32_t)__shfl_xor((int)low, off));
    uint32_t high = low;                             // of all threads
    for (int off = width; off < 64; off *= 2) {
        low = min(low, (uint32_t)__shfl_xor((int)low, off));
        high = max(high, (uint32_t)__shfl_xor((int)high, off));
    }
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        Stat o;
        o.m = __shfl_xor(st.m, off);
        o.s = __shfl_xor(st.s, off);
        o.t = __shfl_xor(st.t, off);
        st.join(o);
    }
    if (lane == 0) stats[wv] = st, lows[wv] = low, highs[wv] = high;
    if (tid == 0) count = 0;
    __syncthreads();
    st = stats[0];
    low = lows[0];
    high = highs[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        st.join(stats[w]);
        low = min(low, lows[w]);
        high = max(high, highs[w]);
    }
    if (topk > 0) {
        if (topk == 1) low = high;
        // past eight groups their least maximum is far below the k-th of all: low's reach, at least
        // topk threads, is halved until few more are left; so it is where a group has no elements at
        // all, and its maximum lets every element through (8192 rows of 540 to 2000, 8 alternatives, bf16: 115
        // us, where ordering all elements took 940)
        if (topk > 8 || (topk > 1 && sp.pieces <= NT - 64))
            for (int step = 0; step < 20 && high - low > 1; ++step) {
                const uint32_t mid = low + (high - low) / 2;
                const int have = __popcll(__ballot(mine >= mid));
                if (lane == 0) reach[step & 1][wv] = have;
                __syncthreads();
                int all = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) all += reach[step & 1][w];
                if (all >= topk) low = mid; else high = mid;
                if (all >= topk && all <= topk + topk / 4) break;
            }
        auto keep = [&](float x, int i) {
            if (order_of(x) < low) return;
            const int at = atomicAdd(&count, 1);
            if (at < kCap) cand[at] = rank_of(x, i);
        };
        if (mine >= low) {
            if (topk > 1 || low == 0xffffffffu) {
                const float least = value_of(max(low, mine == 0xffffffffu ? mine : 0u)); // a maximum passes over NaN
                if (sp.pieces <= NT * U) {
                    sp.singles(keep);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (tid + u * NT < sp.pieces) sp.elements(v[u], tid + u * NT, least, keep);
                } else {
                    sp.each(NT, least, keep);
                }
            } else if (where < 0) {
                const int i = where == -1 ? sp.lo + tid : sp.tail() + tid;
                if (i < sp.hi) keep(ld_io<IO>(sp.row, i), i);
            } else {
                float x[kPer<IO>];
                unpack<IO>(*sp.piece(where), x);
#pragma unroll
                for (int i = 0; i < kPer<IO>; ++i) keep(x[i], sp.first_of(where) + i);
            }
        }
        __syncthreads();
        int n = count;
        __syncthreads();
        if (n > kCap || n < topk) {
            // the topk-th rank, from its highest byte down
            if (tid == 0) prefix = 0;
            int left = topk;
            for (int shift = 48; shift >= 0; shift -= 8) {
                for (int i = tid; i < 256; i += NT) hist[i] = 0;
                __syncthreads();
                const uint64_t top = prefix;
                sp.each(NT, __builtin_nanf(""), [&](float x, int i) {
                    const uint64_t r = rank_of(x, i);
                    if (r >> (shift + 8) == top) atomicAdd(&hist[r >> shift & 255], 1u);
                });
                __syncthreads();
                int digit = 255, above = 0;
                while (above + (int)hist[digit] < left) above += hist[digit--];
                left -= above;
                if (tid == 0) prefix = top << 8 | (uint64_t)digit;
                __syncthreads();
            }
            if (tid == 0) count = 0;
            __syncthreads();
            const uint64_t least = prefix;
            sp.each(NT, __builtin_nanf(""), [&](float x, int i) {
                const uint64_t r = rank_of(x, i);
                if (r >= least) cand[atomicAdd(&count, 1)] = r;
            });
            __syncthreads();
            n = topk;
        }
        if (a.parts > 1) {
            uint64_t* to = a.best + (row * a.parts + part) * topk;
            put_best(cand, n, topk, NT, [&](int i, uint64_t r) { to[i] = r; });
        } else {
            const Row r(st);
            put_best(cand, n, topk, NT, [&](int i, uint64_t x) {
                a.top_logp[row * topk + i] = r.logp(value_of((uint32_t)(x >> 24)));
                a.top_tok[row * topk + i] = index_of(x);
            });
        }
    }
    if (tid == 0) {
        if (a.parts > 1) {
            float* to = a.stat + (row * a.parts + part) * 3;
            to[0] = st.m, to[1] = st.s, to[2] = st.t;
        } else {
            write_row<IO>(a, row, Row(st));
        }
    }
}

// The parts of a row, together.
constexpr int kMaxParts = 16, kMaxJoin = 256;        // parts, and parts times topk
template <int IO>
__global__ void __launch_bounds__(kMaxJoin) score_join(const ScoreArgs a) {
    __shared__ uint64_t cand[kMaxJoin];
    const int64_t row = blockIdx.x;
    Stat st{-FLT_MAX, 0.f, 0.f};
    for (int p = 0; p < a.parts; ++p) {
        const float* from = a.stat + (row * a.parts + p) * 3;
        Stat o;
        o.m = from[0], o.s = from[1], o.t = from[2];
        st.join(o);
    }
    const Row r(st);
    const int n = a.parts * a.topk;
    if ((int)threadIdx.x < n) cand[threadIdx.x] = a.best[row * n + threadIdx.x];
    __syncthreads();
    put_best(cand, n, a.topk, kMaxJoin, [&](int i, uint64_t x) {
        a.top_logp[row * a.topk + i] = r.logp(value_of((uint32_t)(x >> 24)));
        a.top_tok[row * a.topk + i] = index_of(x);
    });
    if (threadIdx.x == 0) write_row<IO>(a, row, r);
}

// ------------------------------------------------------------------ gradient

struct ScoreBackArgs {
    int64_t stride;
    int vocab, topk, parts, part;
    const char* logits;
    const int32_t* tokens;
    const float* lse;
    const float* entropy;
    const float* d_logp;
    const float* d_entropy;
    const int32_t* top_tok;
    const float* d_top;
    char* d_logits;
};

// e^kNever is 0 in fp32: what stands in for ln p below it, near enough that no gradient carries it to infinity.
constexpr float kNever = -200.f;
// From here on lse's own rounding, half a step of it, is 2^-13 of every p and more, and nothing of ln s
// is left in it where a row holds no more than a mask's value.
constexpr float kFarLse = 4096.f;

// m and s of all of a row, by one workgroup of NT threads, in every thread.
template <int IO, int NT>
__device__ Stat whole_row(const Span<IO>& sp) {
    __shared__ Stat stats[NT / 64];
    Stat st{-FLT_MAX, 0.f, 0.f};
    sp.each(NT, __builtin_nanf(""), [&](float x, int) {
        if (x > st.m) st.raise(x);
        st.add(x);
    });
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        Stat o;
        o.m = __shfl_xor(st.m, off);
        o.s = __shfl_xor(st.s, off);
        o.t = __shfl_xor(st.t, off);
        st.join(o);
    }
    if (threadIdx.x % 64 == 0) stats[threadIdx.x / 64] = st;
    __syncthreads();
    st = stats[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) st.join(stats[w]);
    return st;
}

// d x_j = -p_j (sum of the given gradients + d_entropy (ln p_j + entropy)), plus the given
// gradients at their own tokens: these few elements are formed again, whole, by the threads of
// their numbers once the part is written.  Their logits are read before it is, since the
// gradient may take the logits' place.  ln p_j is x_j - lse; of a row with a far lse (kFarLse) the first
// part's workgroup takes all, and has ln p_j = (x_j - m) - ln s from the logits.
template <int IO>
__global__ void __launch_bounds__(256) score_back(const ScoreBackArgs a) {
    constexpr int NT = 256, U = 4, e = IO == GDN_BF16 ? 2 : 4;
    __shared__ int tok[1 + kMaxTop];
    __shared__ float add[1 + kMaxTop];
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts, tid = threadIdx.x;
    const size_t at = (size_t)(row * a.stride) * e;
    Span<IO> sp(a.logits + at, part * a.part, min(a.vocab, (part + 1) * a.part));
    char* out = a.d_logits + at;
    const float lse = a.lse[row];
    const int points = 1 + (a.top_tok ? a.topk : 0);
    int mine = -1;
    float own = 0.f;
    if (tid < points) {
        int t = -1;
        float d = 0.f;
        if (tid > 0) {
            t = a.top_tok[row * a.topk + tid - 1];
            d = a.d_top[row * a.topk + tid - 1];
        } else if (a.tokens) {
            t = a.tokens[row];
            d = a.d_logp[row];
        }
        const bool known = t >= 0 && t < a.vocab;
        tok[tid] = mine = known ? t : -1;
        add[tid] = known ? d : 0.f;
        if (mine < sp.lo || mine >= sp.hi) mine = -1;
        if (mine >= 0) own = ld_io<IO>(sp.row, mine);
    }
    __syncthreads();
    float all = 0.f;
    for (int i = 0; i < points; ++i) all += add[i];
    const float ge = a.d_entropy ? a.d_entropy[row] : 0.f, h = a.d_entropy ? a.entropy[row] : 0.f;
    float from = lse, log_s = 0.f;                   // ln p = (x - from) - log_s
    if (fabsf(lse) >= kFarLse) {
        if (part > 0) return;
        sp = Span<IO>(a.logits + at, 0, a.vocab);
        mine = tid < points ? tok[tid] : -1;
        if (mine >= 0) own = ld_io<IO>(sp.row, mine);
        const Row r(whole_row<IO, NT>(sp));
        from = r.m, log_s = r.log_s;
    }
    auto grad = [&](float x) {
        const float l = (x - from) - log_s, p = __builtin_amdgcn_exp2f(l * kLog2E);
        return -p * (all + ge * (fmaxf(l, kNever) + h));
    };
    if (tid < sp.head) st_io<IO>(out, sp.lo + tid, grad(ld_io<IO>(sp.row, sp.lo + tid)));
    if (tid < sp.hi - sp.tail()) st_io<IO>(out, sp.tail() + tid, grad(ld_io<IO>(sp.row, sp.tail() + tid)));
    u32x4* to = reinterpret_cast<u32x4*>(out + (size_t)(sp.lo + sp.head) * e);
    for (int p0 = tid; p0 < sp.pieces; p0 += NT * U) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p0 + u * NT < sp.pieces) v[u] = *sp.piece(p0 + u * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u * NT >= sp.pieces) break;
            float x[kPer<IO>];
            unpack<IO>(v[u], x);
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (IO == GDN_BF16)
                    w[i] = (uint32_t)bf16_rne(grad(x[2 * i])) | (uint32_t)bf16_rne(grad(x[2 * i + 1])) << 16;
                else
                    w[i] = __float_as_uint(grad(x[i]));
            }
            to[p0 + u * NT] = w;
        }
    }
    __syncthreads();
    if (mine < 0) return;
    float sum = 0.f;
    for (int i = 0; i < points; ++i) {
        if (tok[i] != mine) continue;
        if (i < tid) return;                         // the first of equal tokens writes
        sum += add[i];
    }
    st_io<IO>(out, mine, grad(own) + sum);
}

// ------------------------------------------------------------------ host

bool misaligned(const void* p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
int status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

constexpr int64_t kMaxScoreRows = 1 << 22, kMaxScoreGroups = (1 << 24) - 1;
constexpr int kBackPart = 16384;

int check_dims(const gdn_score_dims* d) {
    if (!d) return GDN_ERR_NULL;
    if (d->io_dtype != GDN_F32 && d->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (d->rows < 0 || d->rows > kMaxScoreRows || d->vocab < 1 || d->vocab > 1 << 24) return GDN_ERR_DIMS;
    if (d->row_stride < d->vocab || d->row_stride > (int64_t)1 << 40) return GDN_ERR_DIMS;
    if (d->topk < 0 || d->topk > kMaxTop || d->topk > d->vocab) return GDN_ERR_DIMS;
    if (d->rows * ((d->vocab + kBackPart - 1) / kBackPart) > kMaxScoreGroups) return GDN_ERR_DIMS;
    return GDN_OK;
}

// Parts of a row, where there are few rows: up to 512 workgroups, of 16384 elements or more each.  (One
// row of 150000 elements, bf16: 8.2 us with one alternative and 14 with eight, against 15.6 and 37
// whole; one of 32000 whole: 6.6 us, against 7.1 in three parts and their join.)
int parts_of(const gdn_score_dims* d) {
    if (d->rows == 0) return 1;
    const int64_t want = 512 / d->rows, most = d->vocab / 16384;
    int64_t parts = std::min<int64_t>({want, most, kMaxParts});
    if (d->topk > 0) parts = std::min<int64_t>(parts, kMaxJoin / d->topk);
    return (int)std::max<int64_t>(parts, 1);
}
// Parts begin at multiples of 64 elements, so that all of a row but the first and last piece is whole.
int part_of(const gdn_score_dims* d, int parts) { return ((d->vocab + parts - 1) / parts + 63) / 64 * 64; }

size_t stat_bytes(const gdn_score_dims* d, int parts) {
    return parts > 1 ? ((size_t)d->rows * parts * 3 * sizeof(float) + 255) / 256 * 256 : 0;
}

int check(std::initializer_list<const void*> need, std::initializer_list<const void*> may) {
    for (const void* p : need)
        if (!p) return GDN_ERR_NULL;
    for (const void* p : need)
        if (misaligned(p)) return GDN_ERR_ALIGN;
    for (const void* p : may)
        if (misaligned(p)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

template <int IO>
hipError_t go(const ScoreArgs& a, int64_t rows, hipStream_t stream) {
    const dim3 grid((uint32_t)(rows * a.parts));
    hipError_t e = launch(score_rows<IO, 512>, grid, dim3(512), 0, stream, a);
    if (e == hipSuccess && a.parts > 1) e = launch(score_join<IO>, dim3((uint32_t)rows), dim3(kMaxJoin), 0, stream, a);
    return e;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_score_workspace_bytes(const gdn_score_dims* dims, size_t* bytes) {
    const int rc = check_dims(dims);
    if (rc) return rc;
    if (!bytes) return GDN_ERR_NULL;
    const int parts = parts_of(dims);
    *bytes = stat_bytes(dims, parts) + (parts > 1 ? (size_t)dims->rows * parts * dims->topk * sizeof(uint64_t) : 0);
    return GDN_OK;
}

int gdn_token_scores(const gdn_score_dims* dims, const void* logits, const int32_t* tokens, float* logp,
                     float* entropy, float* lse, float* top_logp, int32_t* top_tok, void* workspace,
                     hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (dims->rows == 0) return GDN_OK;
    const int parts = parts_of(dims);
    rc = check({logits}, {tokens, logp, entropy, lse, top_logp, top_tok, workspace});
    if (rc) return rc;
    if ((tokens && !logp) || (dims->topk > 0 && (!top_logp || !top_tok)) || (parts > 1 && !workspace)) return GDN_ERR_NULL;
    ScoreArgs a{dims->row_stride, dims->vocab, dims->topk, parts, part_of(dims, parts), (const char*)logits, tokens,
                logp, entropy, lse, top_logp, top_tok, (float*)workspace,
                (uint64_t*)((char*)workspace + stat_bytes(dims, parts))};
    return status_of(dims->io_dtype == GDN_F32 ? go<GDN_F32>(a, dims->rows, stream) : go<GDN_BF16>(a, dims->rows, stream));
}

int gdn_token_scores_backward(const gdn_score_dims* dims, const void* logits, const int32_t* tokens, const float* lse,
                              const float* entropy, const float* d_logp, const float* d_entropy,
                              const int32_t* top_tok, const float* d_top_logp, void* d_logits, hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (dims->rows == 0) return GDN_OK;
    rc = check({logits, lse, d_logits}, {tokens, entropy, d_logp, d_entropy, top_tok, d_top_logp});
    if (rc) return rc;
    if (!tokens != !d_logp || !top_tok != !d_top_logp || (d_entropy && !entropy)) return GDN_ERR_NULL;
    const int parts = (dims->vocab + kBackPart - 1) / kBackPart;
    ScoreBackArgs a{dims->row_stride, dims->vocab, dims->topk, parts, part_of(dims, parts), (const char*)logits, tokens,
                    lse, entropy, d_logp, d_entropy, top_tok, d_top_logp, (char*)d_logits};
    const dim3 grid((uint32_t)(dims->rows * parts));
    return status_of(dims->io_dtype == GDN_F32 ? launch(score_back<GDN_F32>, grid, dim3(256), 0, stream, a)
                                               : launch(score_back<GDN_BF16>, grid, dim3(256), 0, stream, a));
}

}  // extern "C"
