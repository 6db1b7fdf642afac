// attn_rope.hip -- rotary positions of a draft tree's query and key rows.
//
// Pair t of a head's first `rot` coordinates is turned by a = position freq[t] and
// scaled by amp; position = ctx[b] + depth[i].  Every head of a row shares the row's
// angles, so a workgroup forms the cosines and sines of its rows once (in LDS) and
// then streams all heads through them, the first pieces' loads under way meanwhile: the
// kernel is bound by the bytes of q and k, read once and written once (64 trees of 128
// nodes, 36 heads of 128, 151 MB: 23.2 us, 6.5 TB/s).
//
// Angles: position freq is formed in fp64 and reduced to [-pi/4, pi/4] by a two-part
// pi/2 in fp64 (a position of 10^6 turns the fastest pair by 10^6 radians, of which
// fp32 would keep no more than a sixteenth of a radian).  On that interval the Taylor
// sums up to r^15 and r^16 are short of sine and cosine by less than 5e-17.  Their
// products with amp are rounded once, to fp32.
#include "attn_common.hpp"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;                 // one row per wave in the angle phase
constexpr int kRopeUnroll = 4;               // 16-byte pieces in flight per thread

__device__ __forceinline__ void sincos_reduced(double a, double& sn, double& cs) {
    const double n = rint(a * 0.63661977236758134308);           // 2 / pi
    double r = fma(-n, 1.5707963267948965580, a);                // pi / 2, leading 53 bits
    r = fma(-n, 6.1232339957367660359e-17, r);                   // and the next 53
    const int quad = (int)(n - 4.0 * floor(n * 0.25));
    const double x = r * r;
    double s = -1.0 / 1307674368000.0;                           // 1 / 15!
    s = fma(s, x, 1.0 / 6227020800.0);
    s = fma(s, x, -1.0 / 39916800.0);
    s = fma(s, x, 1.0 / 362880.0);
    s = fma(s, x, -1.0 / 5040.0);
    s = fma(s, x, 1.0 / 120.0);
    s = fma(s, x, -1.0 / 6.0);
    s = fma(s * x, r, r);
    double c = 1.0 / 20922789888000.0;                           // 1 / 16!
    c = fma(c, x, -1.0 / 87178291200.0);
    c = fma(c, x, 1.0 / 479001600.0);
    c = fma(c, x, -1.0 / 3628800.0);
    c = fma(c, x, 1.0 / 40320.0);
    c = fma(c, x, -1.0 / 720.0);
    c = fma(c, x, 1.0 / 24.0);
    c = fma(c, x, -0.5);
    c = fma(c, x, 1.0);
    const double ss = (quad & 1) ? c : s, cc = (quad & 1) ? s : c;
    sn = (quad & 2) ? -ss : ss;
    cs = ((quad + 1) & 2) ? -cc : cc;
}

// 16 bytes of elements as fp32 and back.
template <int IO>
struct Piece;
template <>
struct Piece<GDN_F32> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float* f) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
    }
};
template <>
struct Piece<GDN_BF16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b2 v;
            v[0] = (__bf16)f[2 * i];
            v[1] = (__bf16)f[2 * i + 1];
            w[i] = __builtin_bit_cast(uint32_t, v);
        }
        return uint4{w[0], w[1], w[2], w[3]};
    }
};

// Rows leave past the L2: they are read by another launch, and kept there they push out the rows
// still to be read (64 trees of 128 nodes, 36 heads of 128, 151 MB: 38 us; past it 24.6 us).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void put16(char* p, uint4 v) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (u32x4*)p);
}

// Pieces of a head.  kHalf: a rotated piece is 16 bytes of the first coordinates and the
// 16 bytes of their partners; kPairs: 16 bytes of adjacent pairs; the rest is copied, 16
// bytes a piece.  kAny (rot does not divide into 16-byte pieces): one pair or one copied
// coordinate a piece.
enum { kHalf, kPairs, kAny };

template <int IO, int MODE>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, int per_block, int turned, FastDiv pieces,
                                                           FastDiv heads) {
    using P = Piece<IO>;
    constexpr int E = P::E, ES = IO == GDN_F32 ? 4 : 2;
    __shared__ float s_cos[kRopeRows][kMaxHead / 2], s_sin[kRopeRows][kMaxHead / 2];
    __shared__ int s_ok[kRopeRows];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t row0 = (int64_t)blockIdx.x * per_block;
    const int half = a.rot / 2;
    const int H = a.Hq + a.Hk;
    const int total = per_block * H * (int)pieces.d;
    const char* src[kRopeUnroll];
    char* dst[kRopeUnroll];
    uint4 x[kRopeUnroll], y[kRopeUnroll];
    int at[kRopeUnroll], rr[kRopeUnroll];
    // Pieces it0, it0 + kRopeThreads, ... of the workgroup's rows: where they are, and their bytes.
    auto fetch = [&](int it0) {
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int it = it0 + u * kRopeThreads;
            const uint32_t hr = quot(pieces, it);
            const uint32_t r = quot(heads, hr);
            const int c = it - (int)(hr * pieces.d), h = (int)(hr - r * heads.d);
            const int64_t gr = row0 + r;
            rr[u] = it < total && gr < a.rows ? (int)r : -1;
            if (rr[u] < 0) continue;
            const bool isq = h < a.Hq;
            const int hh = isq ? h : h - a.Hq;
            const Rows& in = isq ? a.q : a.k;
            const Rows& out = isq ? a.q_out : a.k_out;
            src[u] = in.p + (gr * in.row + hh * in.head) * ES;
            dst[u] = out.p + (gr * out.row + hh * out.head) * ES;
            at[u] = c;
            if constexpr (MODE != kAny) {
                // element at which the piece begins
                const int e = MODE == kHalf && c >= turned ? a.rot + (c - turned) * E : c * E;
                x[u] = *(const uint4*)(src[u] + e * ES);
                if (MODE == kHalf && c < turned) y[u] = *(const uint4*)(src[u] + (half + e) * ES);
            }
        }
    };
    fetch(tid);                              // under way while the angles are formed
    // Angles: wave w takes row w.
    const int64_t row = row0 + wave;
    if (wave < per_block) {
        int64_t first = -1;
        int b = 0;
        if (row < a.rows) {
            if (a.offsets == nullptr) {
                b = (int)(row / a.N);
                first = b < a.B ? (int64_t)b * a.N : -1;
            } else {
                // the sequence whose rows hold this one: 64 candidates at a time
                for (int s0 = 0; s0 < a.B && first < 0; s0 += 64) {
                    const int s = s0 + lane;
                    const int lo = s < a.B ? a.offsets[s] : -1, hi = s < a.B ? a.offsets[s + 1] : -1;
                    const uint64_t in = __ballot(lo >= 0 && row >= lo && row < hi && (int64_t)hi - lo <= a.N);
                    if (in) {
                        const int at = __ffsll((unsigned long long)in) - 1;
                        b = s0 + at;
                        first = __shfl(lo, at);
                    }
                }
            }
        }
        if (first >= 0) {
            const int dep = a.depth[(int64_t)b * a.N + (row - first)];
            const double pos = (double)a.ctx[b] + (double)dep;
            for (int t = lane; t < half; t += 64) {
                double sn, cs;
                sincos_reduced(pos * a.freq[t], sn, cs);
                s_cos[wave][t] = dep < 0 ? __uint_as_float(0x7fc00000u) : (float)(cs * a.amp);
                s_sin[wave][t] = (float)(sn * a.amp);
            }
            if (lane == 0) s_ok[wave] = dep < 0 ? 2 : 1;
        } else if (lane == 0) {
            s_ok[wave] = 0;
        }
    }
    __syncthreads();
    for (int it0 = tid; it0 < total;) {
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (rr[u] < 0 || s_ok[rr[u]] == 0) continue;
            const float* cs = s_cos[rr[u]];
            const float* sn = s_sin[rr[u]];
            const int c = at[u];
            const bool bad = s_ok[rr[u]] == 2;
            const float nan = __uint_as_float(0x7fc00000u);
            if constexpr (MODE == kAny) {
                const bool turn = c < half;
                const int e0 = !turn ? a.rot + (c - half) : a.layout == GDN_ROPE_HALF ? c : 2 * c;
                const int e1 = a.layout == GDN_ROPE_HALF ? half + c : 2 * c + 1;
                const float f0 = ld_io<IO>(src[u], e0);
                if (turn) {
                    const float f1 = ld_io<IO>(src[u], e1);
                    st_io<IO>(dst[u], e0, f0 * cs[c] - f1 * sn[c]);
                    st_io<IO>(dst[u], e1, f1 * cs[c] + f0 * sn[c]);
                } else {
                    st_io<IO>(dst[u], e0, bad ? nan : f0);
                }
            } else if (c >= turned) {
                const int e = MODE == kHalf ? a.rot + (c - turned) * E : c * E;
                float f[E];
#pragma unroll
                for (int i = 0; i < E; ++i) f[i] = nan;
                put16(dst[u] + e * ES, bad ? P::pack(f) : x[u]);
            } else if constexpr (MODE == kHalf) {
                float f[E], g[E], p[E], q[E];
                P::unpack(x[u], f);
                P::unpack(y[u], g);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float cc = cs[c * E + i], ss = sn[c * E + i];
                    p[i] = f[i] * cc - g[i] * ss;
                    q[i] = g[i] * cc + f[i] * ss;
                }
                put16(dst[u] + c * E * ES, P::pack(p));
                put16(dst[u] + (half + c * E) * ES, P::pack(q));
            } else {
                float f[E], p[E];
                P::unpack(x[u], f);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const float cc = cs[c * (E / 2) + i], ss = sn[c * (E / 2) + i];
                    p[2 * i] = f[2 * i] * cc - f[2 * i + 1] * ss;
                    p[2 * i + 1] = f[2 * i + 1] * cc + f[2 * i] * ss;
                }
                put16(dst[u] + c * E * ES, P::pack(p));
            }
        }
        it0 += kRopeThreads * kRopeUnroll;
        if (it0 < total) fetch(it0);
    }
}

template <int IO>
hipError_t launch_io(const RopeArgs& a, hipStream_t stream) {
    constexpr int E = Piece<IO>::E;
    const int half = a.rot / 2;
    const bool vec_half = a.layout == GDN_ROPE_HALF && half % E == 0;
    const bool vec_pair = a.layout == GDN_ROPE_INTERLEAVED && a.rot % E == 0;
    // Rows of a workgroup: four where that still gives every CU two workgroups, else one, so that a
    // few rows are spread out.
    const int per_block = a.rows >= 2 * 256 * kRopeRows ? kRopeRows : 1;
    int turned, pieces;
    if (vec_half) {
        turned = half / E;
        pieces = turned + (a.d - a.rot) / E;
    } else if (vec_pair) {
        turned = a.rot / E;
        pieces = a.d / E;
    } else {
        turned = half;
        pieces = half + a.d - a.rot;
    }
    const FastDiv fp = fast_div(pieces), fh = fast_div(a.Hq + a.Hk);
    const dim3 grid((unsigned)((a.rows + per_block - 1) / per_block));
    auto* kernel = vec_half ? rope_kernel<IO, kHalf> : vec_pair ? rope_kernel<IO, kPairs> : rope_kernel<IO, kAny>;
    return launch(kernel, grid, dim3(kRopeThreads), 0, stream, a, per_block, turned, fp, fh);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int io, hipStream_t stream) {
    return io == GDN_F32 ? launch_io<GDN_F32>(a, stream) : launch_io<GDN_BF16>(a, stream);
}

}  // namespace gdn
