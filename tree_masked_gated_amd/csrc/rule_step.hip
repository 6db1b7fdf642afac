// rule_step.hip -- the gated delta rule by one token per sequence, on a pool of states.
//
// S' = P + beta (v - P k) k^T with P = g S, and o = S' q = P q + beta (v - P k) (k . q): one pass
// over the state, in fp32, each row of it [d_k] spread over the lanes that read it.  Bound by the
// state's bytes, in and out.  A workgroup of four waves takes kRows rows of a wave's lane groups
// at once, so that each lane has that many 16-byte loads in flight.  64 tokens, 32 heads of 128: 64 us
// for 268 MB, 4.2 TB/s; one token: 7.4 us on the device, the latency of a launch and of two
// dependent reads.
#include "rule_common.hpp"

namespace gdn {
namespace {

constexpr int kRows = 4;

// VEC = 4: columns 4 l .. 4 l + 3 for lane l of LPR; VEC = 1 (d_k not a multiple of 4): l + 64 e.
template <int IO, int VEC, int LPR>
__global__ void __launch_bounds__(256) rule_step(const RuleStepArgs a) {
    constexpr int RW = 64 / LPR;                     // rows of a wave at a time
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane % LPR;
    const int b = blockIdx.y, per = 4 * RW * kRows, blocks = (a.dv + per - 1) / per;
    const int hv = blockIdx.x / blocks, hk = hv / a.group;
    const int first = (blockIdx.x % blocks) * per + wv * RW * kRows + lane / LPR;

    const int s = a.slot ? a.slot[b] : b;
    if (s == -1) return;
    bool good = s >= 0 && s < a.n_states;
    if (good && a.slot)                              // an earlier sequence has it
        for (int j = lane; __any(j < b); j += 64)
            if (__any(j < b && a.slot[j < b ? j : 0] == s)) {
                good = false;
                break;
            }
    float* state = a.state + ((size_t)(good ? s : 0) * a.Hv + hv) * a.dv * a.dk;
    f32x4 x[kRows], k, q;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = first + r * RW;
        x[r] = f32x4{0, 0, 0, 0};
        if (!good || row >= a.dv) continue;
        if constexpr (VEC == 4) {
            if (4 * l < a.dk) x[r] = *reinterpret_cast<const f32x4*>(state + (size_t)row * a.dk + 4 * l);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (l + 64 * e < a.dk) x[r][e] = state[(size_t)row * a.dk + l + 64 * e];
        }
    }
    float kq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = VEC == 4 ? 4 * l + e : l + 64 * e;
        const bool in = c < a.dk;
        k[e] = in ? ld_io<IO>(a.k.p, (size_t)(b * a.k.row + hk * a.k.head + c)) : 0.f;
        q[e] = in ? ld_io<IO>(a.q.p, (size_t)(b * a.q.row + hk * a.q.head + c)) : 0.f;
        kq += k[e] * q[e];
    }
    const float g = a.g[(size_t)b * a.Hv + hv], beta = a.beta[(size_t)b * a.Hv + hv];
    auto sum = [](float v) {                         // over the lanes of a row of the state
#pragma unroll
        for (int off = 1; off < LPR; off *= 2) v += __shfl_xor(v, off);
        return v;
    };
    kq = sum(kq);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = first + r * RW;
        const f32x4 p = g * x[r];
        const float pk = sum(p[0] * k[0] + p[1] * k[1] + p[2] * k[2] + p[3] * k[3]);
        const float pq = sum(p[0] * q[0] + p[1] * q[1] + p[2] * q[2] + p[3] * q[3]);
        if (row >= a.dv) continue;
        const float v = ld_io<IO>(a.v.p, (size_t)(b * a.v.row + hv * a.v.head + row));
        const float u = beta * (v - pk);
        if (l == 0)
            st_io<IO>(a.o.p, (size_t)(b * a.o.row + hv * a.o.head + row), good ? pq + u * kq : __builtin_nanf(""));
        if (!good) continue;
        const f32x4 y = p + u * k;
        if constexpr (VEC == 4) {
            if (4 * l < a.dk) *reinterpret_cast<f32x4*>(state + (size_t)row * a.dk + 4 * l) = y;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (l + 64 * e < a.dk) state[(size_t)row * a.dk + l + 64 * e] = y[e];
        }
    }
}

template <int IO, int VEC, int LPR>
hipError_t go(const RuleStepArgs& a, hipStream_t stream) {
    constexpr int per = 4 * (64 / LPR) * kRows;
    return launch(rule_step<IO, VEC, LPR>, dim3(a.Hv * ((a.dv + per - 1) / per), a.B), dim3(256), 0, stream, a);
}

template <int IO>
hipError_t pick(const RuleStepArgs& a, hipStream_t stream) {
    if (a.dk % 4 != 0) return go<IO, 1, 64>(a, stream);
    return a.dk <= 64 ? go<IO, 4, 16>(a, stream) : a.dk <= 128 ? go<IO, 4, 32>(a, stream) : go<IO, 4, 64>(a, stream);
}

}  // namespace

hipError_t launch_rule_step(const RuleStepArgs& a, int io, hipStream_t stream) {
    return io == GDN_F32 ? pick<GDN_F32>(a, stream) : pick<GDN_BF16>(a, stream);
}

}  // namespace gdn
