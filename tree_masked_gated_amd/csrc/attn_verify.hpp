// attn_verify.hpp -- attention of a draft tree over a paged cache: the kernel, as a
// template on element type, head size and the shape of its tiles.
//
// Mathematics.  The rows of one (sequence, key head) are the n nodes times the group of
// query heads that share the key head.  All of them see the prefix; node i also sees its
// strict ancestors and itself.  The keys of a sequence are one run of ctx + n rows, the
// prefix through the page table, then the tree's own rows; only tiles that reach past ctx
// look at the ancestor bits.  One pass over the keys with a running maximum m (in powers of
// two, scores times scale log2 e), sum l and output acc per row:
//     p = 2^(s - m),  l += p,  acc += p v,
// and where m grows, l and acc are first multiplied by 2^(m_old - m_new).  m may lag behind
// the true maximum by up to kLag: the quotient acc / l does not depend on it, p stays below
// 2^kLag, and most tiles then skip the multiplication.
//
// Tiles.  Scores are formed transposed, S^T = K Q^T, with 16 x 16 matrix instructions: a
// lane then holds four keys of one row, the row's statistics are the lane's own, and the
// packed weights are the second operand of O^T = V^T P^T as they are, provided that V's
// operand lists its keys in the same order.  For bf16 that operand is read from LDS by the
// transposing 64-bit read (four keys of one column per lane); for fp32 its elements are
// single words.
//
// Two ways through the keys, by the rows that share them:
//   - up to 16 rows (next tokens, small trees): the four waves take 32 keys each, from memory to
//     registers to LDS and without a barrier, the next tile's loads under way while one is
//     computed.  Bound by reading the cache: 64 tokens over up to 32k keys, 2.1 GB, 348 to 388 us on
//     different cards, 5.6 to 6.2 TB/s.
//   - more rows: the waves share two or three tiles that go from memory to LDS directly.  They are sent
//     one or two tiles ahead, but not under way for that long: the compiler's waits for page ids count
//     all loads, and take the pieces sent before with them, so that a piece has half a tile's time (256
//     rows) or a tile's to arrive.  128 nodes x 8 query heads per key head over 4k-8k keys, 64 sequences,
//     0.83 TFLOP: 890 us, 929 TFLOP/s.  Matrix instructions fill 44 % of the cycles, vector instructions
//     55 %, and waves wait 32 % of theirs: a weight's scaling, exponential, conversion and sum cost as much
//     as its products.  Every wave reads all of K and V from LDS (256 KB per tile of 64 keys, 1050 of the
//     4700 cycles that a tile takes).  With 256 rows the two waves of a SIMD take turns at the two kinds of
//     work (1005 us where they do not, 953 us where they do, when this was built).
//
// Work.  Tiles of all (sequence, key head, block of rows) form one line, cut into equal
// shares, one per workgroup, so that contexts of very different lengths keep all CUs busy
// to the end without the host knowing the lengths.  A block of rows whose keys were cut
// leaves partial results (m, l, acc in fp32) in the workspace; the workgroup that arrives
// last, by a counter, joins them in the order of the keys, so that results do not depend
// on the order of arrival.  Of the blocks that begin in a share at most the last one is cut, so
// that a share's counters and slots serve batches of any sizes, and calls of different ones
// may follow each other on one workspace.
#pragma once

#include "attn_common.hpp"
#include "attn_schedule.hpp"

namespace gdn {
namespace attn {

constexpr int kCUs = 256, kXcds = 8;
constexpr int kMaxCtx = 0x7fff0000;          // key indexes, whole tiles of them, are 32 bits
constexpr float kLag = 8.0f;
constexpr int kMaxParts = 64;                // pieces of one block of rows
constexpr int kCounterBytes = 18432;         // arrival counters, the workspace's first bytes: zero between calls
constexpr float kLog2e = 1.4426950408889634f;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// IO, D: element type and head size (padded with zeros); RT: tiles of 16 rows per wave; WR waves
// side by side over rows, WK over keys; KT: keys per wave and step; OCC: workgroups per CU.
template <int IO_, int D_, int RT_, int WR_, int WK_, int KT_, int OCC_>
struct Cfg {
    static constexpr int IO = IO_, D = D_, RT = RT_, WR = WR_, WK = WK_, KT = KT_, OCC = OCC_;
    static constexpr int NT = 64 * WR * WK;             // threads
    static constexpr int WAVES = NT / 256 * OCC;        // per SIMD
    static constexpr int ES = IO == GDN_F32 ? 4 : 2;
    static constexpr int E = 16 / ES;                   // elements of a 16-byte piece
    static constexpr int CPR = D / E;                   // pieces of a row
    static constexpr int BM = RT * 16 * WR;             // rows of a workgroup
    static constexpr int KW = KT * WK;                  // keys of a workgroup's step
    static constexpr int TG = 64 * WR;                  // threads that share keys
    static constexpr int NCH = KT * CPR / TG;           // pieces of K (and of V) per thread and step
    static constexpr int KSTEP = TG / CPR;              // keys between a thread's pieces
    static constexpr int STAGES = WR == 1 ? 1 : OCC == 1 && KT * WK * D * ES <= 16384 ? 3 : 2;
    static constexpr int ROWB = D * ES;
    static constexpr int TILEB = KT * ROWB;
    static constexpr int LDS = STAGES * WK * 2 * TILEB;
    static constexpr int DT = D / 16;                   // tiles of 16 columns
    static constexpr int DQ = DT / WK;                  // of these, a wave's share at the end
    static constexpr int KTILES = KT / 16;
    // bf16 elements: a weight's product with V needs a bf16 operand.  Up to 16 rows, which are bound by
    // reading the cache, it is the sum of two, the rounded weight and the rounded rest of it, 2^-16 from the
    // weight at most (next tokens of 64 sequences over up to 32k keys: 348 us with one, 349 us with two).
    // More rows are bound by the work on their weights and take one, 2^-8 from the weight at most (128-node
    // trees of 64 sequences: 915 us with one, 1218 us with two; 128 rows of 64 sequences over 2800 keys 105
    // and 128 us, 64 rows of 128 sequences 134 and 141 us).
    static constexpr int TERMS = IO == GDN_BF16 && WR == 1 ? 2 : 1;
    static constexpr int SLOT = BM * (D + 2) * 4;       // bytes of a partial result
    // The last part of a block stays in registers where a thread's share of it is large (256 rows:
    // 131 KB that are neither written nor read); small ones take one way only.
    static constexpr bool KEEP = RT * DQ >= 16;
    // Time that one more part takes to join, in tiles (88 rows of two sequences over 660 keys: 41 us
    // with 1, 36 us with 1/4; 384 rows over 206 keys 33 and 29; one sequence over 2800 keys 44 and 40).
    // All of these are blocks of 64 rows; blocks of 128 and 256 take the same value untuned.  For those of
    // 256 it is too low: 32 sequences of four such blocks take 19 us without a prefix, 33 us over 64
    // keys and 44 us over 128, which are one and two tiles more for a block.
    static constexpr float PART = IO == GDN_F32 || WR == 1 ? 0.05f : 0.25f;
    // Parts that one workgroup joins.  A token's are small and many: groups of them are joined side by
    // side, then their results (one token over 4k and 32k keys: 23.5 and 46.5 us without groups, 19.8
    // and 40.0 with).  Parts of many rows are few, and a second step costs more than it saves there
    // (one tree of 128 rows over 4k keys: 39 us without, 43 with).
    static constexpr int GROUP = WR == 1 ? 8 : kMaxParts;
    static constexpr int COUNTERS = GROUP < kMaxParts ? 1 + kMaxParts / GROUP : 1;
    static_assert(kCUs * OCC * COUNTERS * 4 <= kCounterBytes, "counters of all shares");
    static_assert(LDS + 4096 <= kMaxLds, "LDS of a workgroup");
    static_assert(TG % CPR == 0 && NCH >= 1, "a thread keeps its piece of the row");
    static_assert(KT % 32 == 0 && DT % WK == 0, "mask words, columns of the joining waves");
};

// Launch parameters that depend on the configuration.
struct Plan {
    int grid;          // workgroups
    int side;          // C: workgroups that take neighbouring blocks of rows over the same keys
    int clusters;      // grid / C
    int max_blocks;    // blocks of rows of the largest tree
    int32_t* arrived;  // [clusters][side][COUNTERS] of the block that is cut at the share's end: its groups,
                       // if any, and the parts of each
    char* slots;       // [grid][2][SLOT]
};

// The place of piece c of a key's row is c ^ swizzle(key).  LDS serves a wave's 16-byte reads of
// K in groups of 16 lanes, keys 0-3 and 12-15 of one piece together with keys 4-11 of the piece
// next to it, and the transposing reads of V in halves, keys 0-7 (8-15) of two neighbouring
// pieces; each must meet all banks once.  For the first the place's lowest bit must not tell
// keys 0-3 and 12-15 from the others, for the second the other bits must tell keys 0-7 apart (and
// 8-15).  fp32 reads V as words of keys 4 g + i of four neighbouring pieces: there the high bits
// tell the g apart.
template <class C>
__device__ __forceinline__ int swizzle(int key) {
    if constexpr (C::IO == GDN_F32) {
        return (((key >> 2) & 3) << 2) | (key & 3);
    } else if constexpr (C::CPR == 8) {      // two keys meet the banks side by side
        const int k = (key >> 1) & 7;
        return (((k & 3) ^ ((k >> 2) << 1)) << 1) | (k >> 2);
    } else {
        const int k = key & 15;
        return (((k & 7) ^ ((k >> 3) << 2)) << 1) | (k >> 3);
    }
}

// Sequence b: its rows, prefix and share of the work.
struct Seq {
    int64_t row0;
    int n, ctx, blocks, tiles, groups;       // groups: ceil(blocks / side)
    bool poison;                             // its rows are NaN
};

template <class C>
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int side, int o0, int o1, int b, int ctx, int status) {
    Seq s;
    s.row0 = (int64_t)b * a.N;
    s.n = a.N;
    if (a.offsets != nullptr) {
        const int64_t n = (int64_t)o1 - o0;
        const bool usable = o0 >= 0 && n >= 0 && n <= a.N;
        s.row0 = usable ? o0 : 0;
        s.n = usable ? (int)n : 0;
    }
    s.poison = status != 0 || ctx < 0 || ctx > kMaxCtx || ctx > (int64_t)a.width * (int64_t)a.page.d;
    s.ctx = s.poison ? 0 : ctx;
    s.blocks = (s.n * a.group + C::BM - 1) / C::BM;
    s.groups = (s.blocks + side - 1) / side;
    s.tiles = s.n == 0 ? 0 : s.poison ? 1 : (int)(((int64_t)s.ctx + s.n + C::KW - 1) / C::KW);
    return s;
}

template <class C>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int side, int b) {
    const int o0 = a.offsets ? a.offsets[b] : 0, o1 = a.offsets ? a.offsets[b + 1] : 0;
    return sequence<C>(a, side, o0, o1, b, a.ctx[b], a.status[b]);
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// 2^x, one instruction.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// Replaces infinities and NaN of a 16-byte piece by zero; whether there were any.
template <int IO>
__device__ __forceinline__ bool clean(uint4& u) {
    uint32_t* w = (uint32_t*)&u;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IO == GDN_F32) {
            const bool x = (w[i] & 0x7f800000u) == 0x7f800000u;
            w[i] = x ? 0u : w[i];
            any |= x;
        } else {
            const bool lo = (w[i] & 0x7f80u) == 0x7f80u, hi = (w[i] & 0x7f800000u) == 0x7f800000u;
            w[i] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
            any |= lo || hi;
        }
    }
    return any;
}

// A wave's view of one (sequence, key head, block of rows) over a run of key tiles.
template <class C>
struct Worker {
    static constexpr int RT = C::RT, DT = C::DT, KTILES = C::KTILES, NCH = C::NCH, ES = C::ES, E = C::E;

    const AttnArgs& a;
    char* lds;
    int* s_flag;                             // [WK]: a tile's V holds infinities or NaN
    int lane, wr, wk, tg;                    // tg: thread within its key group
    int b, h;
    Seq s;

    typename std::conditional<C::IO == GDN_F32, f32x4[C::D / 16], bf16x8[C::D / 32]>::type q[RT];
    f32x4 acc[RT][DT];
    // vectors, not arrays: the compiler keeps them in registers
    float __attribute__((ext_vector_type(RT))) m, l;
    int node[RT];
    uint4 kreg[NCH], vreg[NCH];
    int pid[NCH];
    const char* kbase;                       // this thread's piece of row 0 of page 0
    const char* vbase;
    const int32_t* page_table;
    uint32_t top_page;                       // the largest page id met, as unsigned
    bool bad;
    const bool once;                         // a sequence's keys are read by one block of rows alone

    __device__ __forceinline__ Worker(const AttnArgs& a_, char* lds_, int* flag, bool once_)
        : a(a_), lds(lds_), s_flag(flag), once(once_) {
        const int tid = threadIdx.x;
        lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        wr = wave % C::WR;
        wk = wave / C::WR;
        tg = tid - wk * C::TG;
    }

    // Addresses of the steps that follow are formed anew from here on.  Without this the compiler
    // forms those of every step once, ahead of all of them, and has no registers left for the
    // loop over the prefix.
    __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(lane), "+v"(tg)); }

    __device__ __forceinline__ char* ktile(int stage) const { return lds + (stage * C::WK + wk) * 2 * C::TILEB; }
    __device__ __forceinline__ char* vtile(int stage) const { return ktile(stage) + C::TILEB; }

    __device__ __forceinline__ void begin(int block) {
        fresh();
        const int g = lane >> 4;
        bad = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = -INFINITY;
            l[rt] = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[rt][dt] = zero4();
            const int r = row_of(block, rt);
            const bool real = r < s.n * a.group;
            const int i = (int)quot(a.group_div, r);
            node[rt] = real ? i : -1;
            const char* p = a.q.p + (real ? (s.row0 + i) * a.q.row + (h * a.group + (r - i * a.group)) * a.q.head : 0);
#pragma unroll
            for (int ks = 0; ks < C::CPR / 4; ++ks) {
                const int e = (ks * 4 + g) * E;
                uint4 u = *(const uint4*)(p + (e < a.d ? e * ES : 0));
                if (!real || e >= a.d) u = uint4{0, 0, 0, 0};
                q[rt][ks] = __builtin_bit_cast(typename std::remove_reference<decltype(q[0][0])>::type, u);
            }
        }
    }

    __device__ __forceinline__ int row_of(int block, int rt) const {
        return block * C::BM + (wr * RT + rt) * 16 + (lane & 15);
    }

    // First key of this wave's part of tile t.
    __device__ __forceinline__ int key0(int t) const { return t * C::KW + wk * C::KT; }

    // Page ids of a tile of the prefix.
    __device__ __forceinline__ void fetch_pages(int t) {
        const int j0 = key0(t) + tg / C::CPR;
#pragma unroll
        for (int i = 0; i < NCH; ++i) pid[i] = page_table[quot(a.page, j0 + i * C::KSTEP)];
    }

    // Byte offset of row r of page id in a pool, in pieces of 16.
    static __device__ __forceinline__ uint64_t offset16(const Pool& pool, uint32_t id, uint32_t r) {
        return (uint64_t)id * (uint32_t)pool.page + (uint64_t)r * (uint32_t)pool.row;
    }

    // Keys that one block of rows of the sequence reads do not stay in the L2 (64 tokens over 8k keys
    // each: 218 us, 198 us past it).  Sequences that share pages read them again, and would find them
    // there; the host does not know of them (the same where fours share their pages: 170 us, 183 us
    // past it; 32 rows over 4k keys 99 and 122 us).
    static __device__ __forceinline__ uint4 get16_once(const char* p) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4*)p));
    }

    // Loads a tile of the prefix into registers, through the page ids fetched before.
    __device__ __forceinline__ void load(int t) {
        const int j0 = key0(t) + tg / C::CPR;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t j = j0 + i * C::KSTEP;
            const uint32_t r = j - quot(a.page, j) * a.page.d;
            top_page = max(top_page, (uint32_t)pid[i]);
            const uint32_t id = min((uint32_t)pid[i], (uint32_t)a.n_pages - 1u);
            kreg[i] = get16_once(kbase + (offset16(a.kp, id, r) << 4));
            vreg[i] = get16_once(vbase + (offset16(a.vp, id, r) << 4));
        }
    }

    // The same for a tile that reaches the tree's own rows, or past them.
    __device__ __forceinline__ void load_mixed(int t) {
        const int c = tg % C::CPR;
        const int j0 = key0(t) + tg / C::CPR;
        const int64_t in_row = c * E < a.d ? c * 16 : 0;
        bool any = false;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int j = j0 + i * C::KSTEP;
            kreg[i] = vreg[i] = uint4{0, 0, 0, 0};
            if (j < s.ctx) {
                const uint32_t pg = quot(a.page, j);
                const uint32_t at = page_table[pg];
                top_page = max(top_page, at);
                const uint32_t id = min(at, (uint32_t)a.n_pages - 1u), r = j - pg * a.page.d;
                kreg[i] = *(const uint4*)(kbase + (offset16(a.kp, id, r) << 4));
                vreg[i] = *(const uint4*)(vbase + (offset16(a.vp, id, r) << 4));
            } else if (j < s.ctx + s.n) {
                const int64_t r = s.row0 + (j - s.ctx);
                kreg[i] = *(const uint4*)(a.k.p + h * a.k.head + in_row + r * a.k.row);
                vreg[i] = *(const uint4*)(a.v.p + h * a.v.head + in_row + r * a.v.row);
            }
            // A zero weight times an infinity is no zero: what is not finite is kept out of the
            // product and added to the rows that see it (spread()).
            any |= clean<C::IO>(vreg[i]);
        }
        if (any) s_flag[wk] = 1;
    }

    // Registers to LDS.
    __device__ __forceinline__ void store(int stage) {
        char* kt = ktile(stage);
        char* vt = vtile(stage);
        const int c = tg % C::CPR, k0 = tg / C::CPR;
        const bool pad = c * E >= a.d;       // columns past d: the query's are zero, the key's must be finite
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int key = k0 + i * C::KSTEP;
            if (pad) kreg[i] = uint4{0, 0, 0, 0};
            const int at = key * C::ROWB + ((c ^ swizzle<C>(key)) * 16);
            *(uint4*)(kt + at) = kreg[i];
            *(uint4*)(vt + at) = vreg[i];
        }
    }

    // Bits of the keys of block kb (32 keys from key j0 + 32 kb on) that row rt sees.
    __device__ __forceinline__ uint32_t seen(int j0, int kb, int rt) const {
        const int x = j0 + 32 * kb - s.ctx;             // node index of the first key
        const int w0 = x >> 5, sh = x & 31;
        const uint32_t lo = seen_word(w0, rt), hi = seen_word(w0 + 1, rt);
        return sh == 0 ? lo : (lo >> sh) | (hi << (32 - sh));
    }
    __device__ __forceinline__ uint32_t seen_word(int w, int rt) const {
        if (w < 0) return 0xffffffffu;                  // the prefix
        if (node[rt] < 0 || w * 32 >= s.n) return 0u;
        uint32_t x = a.anc[((int64_t)b * a.N + node[rt]) * a.words + w];
        if ((node[rt] >> 5) == w) x |= 1u << (node[rt] & 31);
        const int left = s.n - w * 32;
        return left < 32 ? x & ((1u << left) - 1u) : x;
    }

    // Scores of a tile's keys, raw products.
    __device__ __forceinline__ void scores(const char* kt, f32x4 (&sc)[RT][KTILES]) const {
        const int g = lane >> 4, c16 = lane & 15;
#pragma unroll
        for (int x = 0; x < KTILES; ++x) {
            const char* row = kt + c16 * C::ROWB + x * 16 * C::ROWB;
            const int z = swizzle<C>(c16);              // of key 16 x + c16: its low four bits count
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) sc[rt][x] = zero4();
#pragma unroll
            for (int ks = 0; ks < C::CPR / 4; ++ks) {
                const uint4 u = *(const uint4*)(row + ((ks * 4 + g) ^ z) * 16);
                if constexpr (C::IO == GDN_F32) {
                    const f32x4 kf = __builtin_bit_cast(f32x4, u);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            sc[rt][x] = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[e], q[rt][ks][e], sc[rt][x], 0, 0, 0);
                } else {
                    const bf16x8 kf = __builtin_bit_cast(bf16x8, u);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        sc[rt][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[rt][ks], sc[rt][x], 0, 0, 0);
                }
            }
        }
    }

    // Running maximum, moved only where it lags too far.
    __device__ __forceinline__ void raise(const f32x4 (&sc)[RT][KTILES]) {
        const float scale = a.scale * kLog2e;
        float top[RT];
        bool move = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            top[rt] = -INFINITY;
#pragma unroll
            for (int x = 0; x < KTILES; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) top[rt] = fmaxf(top[rt], sc[rt][x][i]);
            top[rt] *= scale;
            move |= top[rt] > m[rt] + kLag;
        }
        if (__any(move)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float x = top[rt];
                x = fmaxf(x, __shfl_xor(x, 16));
                x = fmaxf(x, __shfl_xor(x, 32));
                x = fmaxf(x, m[rt]);
                const float f = x == m[rt] ? 1.f : exp2_fast(m[rt] - x);
                m[rt] = x;
                l[rt] *= f;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= f;
            }
        }
    }

    // Weights of a tile's keys from their scores, and their sum.
    typedef typename std::conditional<C::IO == GDN_F32, f32x4, bf16x8>::type Weights;
    static constexpr int PX = C::IO == GDN_F32 ? KTILES : KTILES / 2, NP = PX * C::TERMS;
    __device__ __forceinline__ void weigh(f32x4 (&sc)[RT][KTILES], Weights (&p)[RT][NP]) {
        const float scale = a.scale * kLog2e;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float base = m[rt] == -INFINITY ? 0.f : m[rt];
#pragma unroll
            for (int x = 0; x < KTILES; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[rt][x][i] = exp2_fast(fmaf(sc[rt][x][i], scale, -base));
            if constexpr (C::IO == GDN_F32) {
#pragma unroll
                for (int x = 0; x < KTILES; ++x) {
                    p[rt][x] = sc[rt][x];
                    l[rt] += (sc[rt][x][0] + sc[rt][x][1]) + (sc[rt][x][2] + sc[rt][x][3]);
                }
            } else {
                // l sums the terms that the product takes, so that the weights' quotients add up to
                // one and a row that sees one key gets that key's value exactly.
                const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
                for (int x = 0; x < KTILES / 2; ++x) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const f32x4& src = sc[rt][2 * x + (i >> 2)];
                        bf16x2 v;
                        v[0] = (__bf16)src[i & 3];
                        v[1] = (__bf16)src[(i & 3) + 1];
                        l[rt] = __builtin_amdgcn_fdot2_f32_bf16(v, one, l[rt], false);
                        p[rt][x][i] = v[0];
                        p[rt][x][i + 1] = v[1];
                        if constexpr (C::TERMS == 2) {
                            bf16x2 rest;
                            rest[0] = (__bf16)(src[i & 3] - (float)v[0]);
                            rest[1] = (__bf16)(src[(i & 3) + 1] - (float)v[1]);
                            l[rt] = __builtin_amdgcn_fdot2_f32_bf16(rest, one, l[rt], false);
                            p[rt][PX + x][i] = rest[0];
                            p[rt][PX + x][i + 1] = rest[1];
                        }
                    }
                }
            }
        }
    }

    // acc += weights times a tile's values.
    __device__ __forceinline__ void values(const char* vt, const Weights (&p)[RT][NP]) {
        const int g = lane >> 4, c16 = lane & 15;
        if constexpr (C::IO == GDN_F32) {
#pragma unroll
            for (int x = 0; x < KTILES; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const char* row = vt + 4 * g * C::ROWB + (x * 16 + i) * C::ROWB;
                    const int z = swizzle<C>(4 * g + i);
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const float v = *(const float*)(row + ((dt * 4 + (c16 >> 2)) ^ z) * 16 + (c16 & 3) * 4);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            acc[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, p[rt][x][i], acc[rt][dt], 0, 0, 0);
                    }
                }
        } else {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
#pragma unroll
            for (int x = 0; x < KTILES / 2; ++x) {
                // lane (row of the read c16 / 4, columns 4 (c16 % 4) ..): keys 4g + c16 / 4 of both halves
                const int key = 4 * g + (c16 >> 2);
                const char* row = vt + key * C::ROWB + (c16 & 1) * 8 + x * 32 * C::ROWB;
                const int z = swizzle<C>(key);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    const int c = dt * 2 + ((c16 >> 1) & 1);
                    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(row + (c ^ z) * 16));
                    const s16x4 hi =
                        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(row + 16 * C::ROWB + (c ^ z) * 16));
                    bf16x8 v;
                    const bf16x4 vl = __builtin_bit_cast(bf16x4, lo), vh = __builtin_bit_cast(bf16x4, hi);
                    v = __builtin_shufflevector(vl, vh, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int y = x; y < NP; y += PX)
                            acc[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[rt][y], acc[rt][dt], 0, 0, 0);
                }
            }
        }
    }

    // values() and the next tile's scores() as one run of 2 RT products per LDS fragment: the
    // fragments 0 .. kPv - 1 are those of V, the others those of K.
    static constexpr int kPv = KTILES / 2 * DT, kFrags = kPv + KTILES * (C::CPR / 4);
    static constexpr int kEarly = 5;         // fragments read ahead: their latency in products
    __device__ __forceinline__ bf16x8 fragment(int u, const char* vt, const char* kt) const {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int g = lane >> 4, c16 = lane & 15;
        if (u < kPv) {
            // lane (row of the read c16 / 4, columns 4 (c16 % 4) ..): keys 4g + c16 / 4 of both halves
            const int key = 4 * g + (c16 >> 2), c = u % DT * 2 + ((c16 >> 1) & 1);
            const char* at = vt + (u / DT * 32 + key) * C::ROWB + (c16 & 1) * 8 + (c ^ swizzle<C>(key)) * 16;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * C::ROWB));
            return __builtin_shufflevector(__builtin_bit_cast(bf16x4, lo), __builtin_bit_cast(bf16x4, hi), 0, 1, 2,
                                           3, 4, 5, 6, 7);
        }
        const int x = (u - kPv) % KTILES, ks = (u - kPv) / KTILES;
        return *(const bf16x8*)(kt + (x * 16 + c16) * C::ROWB + ((ks * 4 + g) ^ swizzle<C>(c16)) * 16);
    }
    __device__ __forceinline__ void products(const char* vt, const char* kt, const Weights (&p)[RT][NP],
                                             bf16x8 (&f)[kFrags], f32x4 (&sc)[RT][KTILES]) {
#pragma unroll
        for (int u = 0; u < kFrags; ++u) {
            if (u + kEarly < kFrags) f[u + kEarly] = fragment(u + kEarly, vt, kt);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if (u < kPv) {
                    f32x4& to = acc[rt][u % DT];
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[u], p[rt][u / DT], to, 0, 0, 0);
                } else {
                    const int x = (u - kPv) % KTILES, ks = (u - kPv) / KTILES;
                    if (ks == 0) sc[rt][x] = zero4();
                    sc[rt][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[u], q[rt][ks], sc[rt][x], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0x6);     // only addresses may move
        }
    }

    // A tile in LDS, all at once.
    template <bool MIXED>
    __device__ __forceinline__ void compute(int t, int stage) {
        f32x4 sc[RT][KTILES];
        scores(ktile(stage), sc);
        const int j0 = key0(t);
        if constexpr (MIXED) {
            const int g = lane >> 4;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
                for (int kb = 0; kb < C::KT / 32; ++kb) {
                    const uint32_t bits = seen(j0, kb, rt) >> (4 * g);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((bits >> (16 * x + i)) & 1u)) sc[rt][2 * kb + x][i] = -INFINITY;
                }
            }
        }
        raise(sc);
        Weights p[RT][NP];
        weigh(sc, p);
        values(vtile(stage), p);
        if constexpr (MIXED) {
            if (s_flag[wk] != 0) spread(j0);
        }
    }

    // Waves that share tiles: the pieces of a tile go from the pools to LDS without passing
    // through registers.  A wave's 64 pieces land side by side, so that thread tg fills the place
    // tg + i TG of the tile and fetches the piece that belongs there.
    struct Ahead {
        uint64_t k[NCH], v[NCH];             // offsets in pieces of 16 bytes from the pools' data
    };
    __device__ __forceinline__ int piece_at(int i) const {
        return (tg % C::CPR) ^ swizzle<C>(tg / C::CPR + i * C::KSTEP);
    }
    __device__ __forceinline__ Ahead locate(int t, const int (&ids)[NCH]) {
        const int j0 = key0(t) + tg / C::CPR;
        Ahead at;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t j = j0 + i * C::KSTEP;
            const uint32_t r = j - quot(a.page, j) * a.page.d;
            top_page = max(top_page, (uint32_t)ids[i]);
            const uint32_t id = min((uint32_t)ids[i], (uint32_t)a.n_pages - 1u);
            at.k[i] = offset16(a.kp, id, r) + piece_at(i);
            at.v[i] = offset16(a.vp, id, r) + piece_at(i);
        }
        return at;
    }
    __device__ __forceinline__ void to_lds(const char* base, const uint64_t (&at)[NCH], char* tile) const {
        const uint32_t to = __builtin_amdgcn_readfirstlane(
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)tile + wr * 1024);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const char* from = base + (at[i] << 4);
            if (piece_at(i) * E < a.d) {     // LDS holds zeros where a row has ended
                // bound by memory where the rows are few: 128 sequences, 64 rows over 2800 keys, 152 us,
                // 135 us past the L2 (not with heads of 256: 454 us, 480 us)
                if (C::WR < 8 && C::D <= 128 && once)
                    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
                                 :: "s"(to + i * C::TG * 16), "v"(from) : "memory");
                else
                    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                                 :: "s"(to + i * C::TG * 16), "v"(from) : "memory");
            }
        }
    }
    // All but the newest `later` pieces that this thread sent to LDS have arrived.  Loads that the
    // compiler places among them only make the wait longer.
    template <int later>
    static __device__ __forceinline__ void wait() {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(later) : "memory");
    }
    // A barrier between the halves of a tile.  This wave's reads of LDS have returned; what it has
    // under way to LDS is waited for elsewhere.
    static __device__ __forceinline__ void turn() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // Tiles [t0, full), in the order of attn_schedule.hpp.  While the values of tile t are added, the
    // scores of t + 1 are formed: both products and the exponentials between them are independent
    // and fill each other's gaps.
    struct Walk {
        Worker& w;
        const char* const kb;                // row 0 of page 0
        const char* const vb;
        Ahead old, at;
        int ids[NCH];
        f32x4 sc[RT][KTILES];
        Weights p[RT][NP];
        bf16x8 f[kFrags];

        __device__ __forceinline__ void fetch(int t) { w.fetch_pages(t); }
        __device__ __forceinline__ void keep() {
#pragma unroll
            for (int i = 0; i < NCH; ++i) ids[i] = w.pid[i];
        }
        __device__ __forceinline__ void locate(int t) {
            old = at;
            at = w.locate(t, w.pid);
        }
        __device__ __forceinline__ void locate_kept(int t) {
            old = at;
            at = w.locate(t, ids);
        }
        __device__ __forceinline__ void send_k(int slot) { w.to_lds(kb, at.k, w.ktile(slot)); }
        __device__ __forceinline__ void send_v(int slot) { w.to_lds(vb, old.v, w.vtile(slot)); }
        // Sends of this thread, all but those of one tile's K (and V), have arrived.
        __device__ __forceinline__ void wait_k() const {
            if (w.a.d < C::D)
                wait<0>();
            else
                wait<NCH>();
        }
        __device__ __forceinline__ void wait_sent(bool all) const {
            if (all || w.a.d < C::D)
                wait<0>();
            else
                wait<2 * NCH>();
        }
        __device__ __forceinline__ void barrier() const { __syncthreads(); }
        __device__ __forceinline__ void turn() const { Worker::turn(); }
        __device__ __forceinline__ void scores(int slot) { w.scores(w.ktile(slot), sc); }
        __device__ __forceinline__ void early(int here, int next) {
#pragma unroll
            for (int u = 0; u < kEarly; ++u) f[u] = w.fragment(u, w.vtile(here), w.ktile(next));
        }
        __device__ __forceinline__ void weights() {
            w.raise(sc);
            w.weigh(sc, p);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int x = 0; x < NP; ++x) asm volatile("" : "+v"(p[rt][x]));   // formed by here
        }
        __device__ __forceinline__ void products(int here, int next) {
            __builtin_amdgcn_s_setprio(1);
            w.products(w.vtile(here), w.ktile(next), p, f, sc);
            __builtin_amdgcn_s_setprio(0);
        }
        __device__ __forceinline__ void tile(int here, int next) {
            w.raise(sc);
            f32x4 sc1[RT][KTILES];
            w.scores(w.ktile(next), sc1);
            w.weigh(sc, p);
            w.values(w.vtile(here), p);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int x = 0; x < KTILES; ++x) sc[rt][x] = sc1[rt][x];
        }
        __device__ __forceinline__ void finish(int here) {
            w.raise(sc);
            w.weigh(sc, p);
            w.values(w.vtile(here), p);
        }
    };
    __device__ __forceinline__ void run_prefix(int t0, int full) {
        if (a.d < C::D) {
            for (int i = wk * C::TG + tg; i < C::LDS / 16; i += C::NT) ((uint4*)lds)[i] = uint4{0, 0, 0, 0};
            __syncthreads();
        }
        Walk o{*this, a.kp.p + (int64_t)h * a.kp.head, a.vp.p + (int64_t)h * a.vp.head};
        if constexpr (C::WR == 8)
            walk_in_turns<C::STAGES>(t0, full, wr < 4, o);   // the two waves of a SIMD
        else
            walk_in_step<C::STAGES>(t0, full, o);
    }

    // Adds the infinities and NaN of this part's values to the rows that see them (a cold path: one
    // key after the other, a few registers, so that it costs the main loop none).
    __device__ __forceinline__ void spread(int j0) {
        const int g = lane >> 4;
#pragma unroll 1
        for (int kb = 0; kb < C::KT / 32; ++kb) {
            uint32_t bits[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) bits[rt] = seen(j0, kb, rt);
#pragma unroll 1
            for (int kk = 0; kk < 32; ++kk) {
                const int j = j0 + kb * 32 + kk;
                if (j >= s.ctx + s.n) break;
                const char* vp;
                if (j < s.ctx) {
                    const int pg = (int)quot(a.page, j);
                    const int id = a.table[(int64_t)b * a.width + pg];
                    if ((uint32_t)id >= (uint32_t)a.n_pages) continue;
                    vp = a.vp.p + (int64_t)h * a.vp.head + (offset16(a.vp, id, j - pg * (int)a.page.d) << 4);
                } else {
                    vp = a.v.p + (s.row0 + (j - s.ctx)) * a.v.row + h * a.v.head;
                }
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    const int e = dt * 16 + 4 * g;
                    const char* at = vp + (e < a.d ? e : 0) * ES;      // columns past d are not written
                    f32x4 v;
                    if constexpr (C::IO == GDN_F32)
                        v = *(const f32x4*)at;
                    else
                        v = __builtin_convertvector(*(const bf16x4*)at, f32x4);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[rt][dt][i] += ((bits[rt] >> kk) & 1u) && nonfinite(v[i]) ? v[i] : 0.f;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    // Tiles [t0, t1) of the block: those of the prefix alone, the next one's loads under way while
    // one is computed, then the few that reach the tree's own rows, one after the other.
    __device__ __forceinline__ void run(int t0, int t1) {
        fresh();
        const int c = tg % C::CPR;
        const int in_row = c * E < a.d ? c * 16 : 0;
        kbase = a.kp.p + (int64_t)h * a.kp.head + in_row;
        vbase = a.vp.p + (int64_t)h * a.vp.head + in_row;
        page_table = a.table + (int64_t)b * a.width;
        top_page = 0;
        __syncthreads();                     // the last run's LDS is done with
        const int full = min(t1, s.ctx / C::KW);
        int t = t0;
        if (t < full) {
            if constexpr (C::WR > 1) {
                run_prefix(t, full);
                t = full;
            } else {
                fetch_pages(t);
                load(t);
                if (t + 1 < full) fetch_pages(t + 1);
                store(0);
                for (; t + 1 < full; ++t) {
                    load(t + 1);
                    fetch_pages(min(t + 2, full - 1));
                    compute<false>(t, 0);
                    store(0);
                }
                compute<false>(t, 0);
                ++t;
            }
        }
        fresh();
        for (; t < t1; ++t) {
            __syncthreads();
            if (threadIdx.x < C::WK) s_flag[threadIdx.x] = 0;
            __syncthreads();
            load_mixed(t);
            store(0);
            __syncthreads();
            compute<true>(t, 0);
        }
        bad = top_page >= (uint32_t)a.n_pages;
    }

    // Joins the waves that split the keys.  Afterwards wave wk holds the columns of its share in
    // acc[rt][0 .. DQ), and every wave has the rows' m and l.
    __device__ __forceinline__ void join_waves() {
        fresh();
        const int c16 = lane & 15;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            l[rt] += __shfl_xor(l[rt], 16);
            l[rt] += __shfl_xor(l[rt], 32);
        }
        bad = __syncthreads_or(bad) != 0;
        if constexpr (C::WK > 1) {
            float* ml = (float*)lds;                    // [WK][WR RT 16][2]
            constexpr int ROWS = C::WR * RT * 16;
            const int r0 = wr * RT * 16 + c16;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                if (lane < 16) {
                    ml[(wk * ROWS + r0 + rt * 16) * 2] = m[rt];
                    ml[(wk * ROWS + r0 + rt * 16) * 2 + 1] = l[rt];
                }
            __syncthreads();
            float w[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float mm[C::WK], top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int k = 0; k < C::WK; ++k) {
                    mm[k] = ml[(k * ROWS + r0 + rt * 16) * 2];
                    top = fmaxf(top, mm[k]);
                }
#pragma unroll
                for (int k = 0; k < C::WK; ++k)
                    sum += ml[(k * ROWS + r0 + rt * 16) * 2 + 1] * weight(mm[k], top);
                w[rt] = weight(m[rt], top);
                m[rt] = top;
                l[rt] = sum;
            }
            f32x4* part = (f32x4*)(lds + C::WK * ROWS * 8);   // [WK][WR][RT][DQ][64]
            f32x4 mine[RT][C::DQ];
#pragma unroll
            for (int k = 0; k < C::WK; ++k) {
                if (k > 0) __syncthreads();
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int dq = 0; dq < C::DQ; ++dq)
                        part[(((wk * C::WR + wr) * RT + rt) * C::DQ + dq) * 64 + lane] = acc[rt][k * C::DQ + dq] * w[rt];
                __syncthreads();
                if (wk == k) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int dq = 0; dq < C::DQ; ++dq) {
                            f32x4 x = zero4();
#pragma unroll
                            for (int j = 0; j < C::WK; ++j)
                                x += part[(((j * C::WR + wr) * RT + rt) * C::DQ + dq) * 64 + lane];
                            mine[rt][dq] = x;
                        }
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int dq = 0; dq < C::DQ; ++dq) acc[rt][dq] = mine[rt][dq];
        }
        if (bad) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) l[rt] = __uint_as_float(0x7fc00000u);
        }
    }

    // 2^(m - top) of partial results; those of no visible key (m = -inf) weigh nothing.
    static __device__ __forceinline__ float weight(float m, float top) {
        return m == -INFINITY ? 0.f : exp2_fast(m - top);
    }

    // Rows of the block to o: acc[rt][0 .. DQ) / l.
    __device__ __forceinline__ void write(int block, bool poison) {
        fresh();
        const int g = lane >> 4;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row_of(block, rt);
            if (r >= s.n * a.group) continue;
            const int i = (int)quot(a.group_div, r);
            char* p = a.o.p + (s.row0 + i) * a.o.row + (h * a.group + (r - i * a.group)) * a.o.head;
            const float inv = 1.f / l[rt];
#pragma unroll
            for (int dq = 0; dq < C::DQ; ++dq) {
                const int e = (wk * C::DQ + dq) * 16 + 4 * g;
                if (e >= a.d) continue;
                f32x4 x = acc[rt][dq] * inv;
                if (poison) x = f32x4{1.f, 1.f, 1.f, 1.f} * __uint_as_float(0x7fc00000u);
                if constexpr (C::IO == GDN_F32)
                    *(f32x4*)(p + e * ES) = x;
                else
                    *(bf16x4*)(p + e * ES) = __builtin_convertvector(x, bf16x4);
            }
        }
    }

    // Partial results in the lanes' own order: [WR RT][DT][64] columns, then m and l by row.
    __device__ __forceinline__ f32x4* slot_acc(char* slot, int rt, int dq) const {
        return (f32x4*)slot + ((wr * RT + rt) * DT + wk * C::DQ + dq) * 64 + lane;
    }
    __device__ __forceinline__ float* slot_ml(char* slot, int rt) const {
        return (float*)(slot + C::BM * C::D * 4) + ((wr * RT + rt) * 16 + (lane & 15)) * 2;
    }
    // They pass between XCDs, whose L2 caches do not see each other's lines.  Their stores and
    // loads are relaxed atomics of device scope, which go past these caches one by one; fences of
    // that scope would write back and drop whole caches, once per wave (token steps of 64
    // sequences over 128 keys: 70 us with fences).
    static __device__ __forceinline__ void put(f32x4* p, f32x4 v) {
        const uint64_t lo = __builtin_bit_cast(uint64_t, __builtin_shufflevector(v, v, 0, 1));
        const uint64_t hi = __builtin_bit_cast(uint64_t, __builtin_shufflevector(v, v, 2, 3));
        __hip_atomic_store((uint64_t*)p, lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store((uint64_t*)p + 1, hi, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    static __device__ __forceinline__ f32x2 get2(const void* p) {
        return __builtin_bit_cast(
            f32x2, __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    }
    static __device__ __forceinline__ f32x4 get(const f32x4* p) {
        return __builtin_shufflevector(get2(p), get2((const uint64_t*)p + 1), 0, 1, 2, 3);
    }
    __device__ __forceinline__ void save(char* slot) const {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int dq = 0; dq < C::DQ; ++dq) put(slot_acc(slot, rt, dq), acc[rt][dq]);
            if (wk == 0 && lane < 16)
                __hip_atomic_store((uint64_t*)slot_ml(slot, rt), __builtin_bit_cast(uint64_t, f32x2{m[rt], l[rt]}),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        // Stores that have returned are at the device's coherence point: what a thread does after
        // the next barrier comes after them.
        __builtin_amdgcn_s_waitcnt(0);
    }
    // Parts 0 .. n - 1 of a block, in the order of their keys; slot_of(i) is part i's place.  With
    // KEEP part `mine` is in this workgroup's registers.
    template <class F>
    __device__ __forceinline__ void join_parts(int n, int mine, F slot_of) {
        fresh();
        // parts whose loads are in flight together
        constexpr int U = C::DQ >= 8 ? 1 : 8 / C::DQ;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const f32x2 own_ml = f32x2{m[rt], l[rt]};
            f32x4 own[C::DQ];
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int dq = 0; dq < C::DQ; ++dq) {
                own[dq] = acc[rt][dq];
                acc[rt][dq] = zero4();
            }
            for (int i0 = 0; i0 < n; i0 += U) {
                f32x2 ml[U];
                f32x4 x[U][C::DQ];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = min(i0 + u, n - 1);
                    if (C::KEEP && i == mine) {
                        ml[u] = own_ml;
#pragma unroll
                        for (int dq = 0; dq < C::DQ; ++dq) x[u][dq] = own[dq];
                        continue;
                    }
                    char* slot = slot_of(i);
                    ml[u] = get2(slot_ml(slot, rt));
#pragma unroll
                    for (int dq = 0; dq < C::DQ; ++dq) x[u][dq] = get(slot_acc(slot, rt, dq));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i0 + u >= n) break;             // its columns may be infinite: not even times zero
                    const float next = fmaxf(top, ml[u][0]);
                    const float w0 = weight(top, next), w1 = weight(ml[u][0], next);
                    top = next;
                    sum = sum * w0 + ml[u][1] * w1;
#pragma unroll
                    for (int dq = 0; dq < C::DQ; ++dq) acc[rt][dq] = acc[rt][dq] * w0 + x[u][dq] * w1;
                }
            }
            m[rt] = top;
            l[rt] = sum;
        }
    }
};

template <class C>
__global__ __launch_bounds__(C::NT, C::WAVES) void attn_kernel(AttnArgs a, Plan plan) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ int64_t s_pre[C::NT];
    __shared__ int64_t s_part[C::NT / 64];
    __shared__ int s_max[C::NT / 64];
    __shared__ int s_flag[2 * 4];
    __shared__ int s_pick, s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // Neighbouring shares on one XCD, whose L2 then holds the keys that they have in common.
    const int per = plan.grid / kXcds;
    const int logical = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
    const int cluster = logical / plan.side, member = logical % plan.side;
    if (cluster >= plan.clusters) return;

    // The line of tiles: sequence b owns Hk groups tiles of it.  Its length, and the longest block.
    int64_t total = 0;
    int longest = 0;
    for (int b0 = 0; b0 < a.B; b0 += C::NT) {
        int64_t x = 0;
        int t = 0;
        if (b0 + tid < a.B) {
            const Seq s = load_seq<C>(a, plan.side, b0 + tid);
            t = s.tiles;
            x = (int64_t)a.Hk * s.groups * s.tiles;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t y = __shfl_up(x, o);
            if (lane >= o) x += y;
            t = max(t, __shfl_xor(t, o));
        }
        if (lane == 63) s_part[wave] = x;
        if (lane == 0) s_max[wave] = t;
        __syncthreads();
        int64_t base = total;
#pragma unroll
        for (int w = 0; w < C::NT / 64; ++w) {
            if (w < wave) base += s_part[w];
            total += s_part[w];
            longest = max(longest, s_max[w]);
        }
        s_pre[tid] = base + x;               // kept where one round covers the batch
        __syncthreads();
    }
    // Shares of a block of n tiles in shares of s take s tiles' time and then n / s parts' to join;
    // a workgroup that would otherwise idle is not worth a part below s = sqrt(n PART).
    const int least = max((longest + kMaxParts - 2) / (kMaxParts - 1), (int)__fsqrt_rn((float)longest * C::PART));
    const int64_t share = max((total + plan.clusters - 1) / plan.clusters, (int64_t)least);
    int64_t at = cluster * share;
    const int64_t end = min(total, at + share);
    if (at >= end) return;

    // The sequence in which the share begins, and where that sequence begins on the line.
    int b = 0;
    int64_t start = 0;
    if (a.B <= C::NT) {
        const int n = __popcll(__ballot(tid < a.B && s_pre[tid] <= at));
        if (lane == 0) s_max[wave] = n;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < C::NT / 64; ++w) b += s_max[w];
        start = b > 0 ? s_pre[b - 1] : 0;
    } else {
        // many sequences: walk the line again, a round at a time
        if (tid == 0) s_pick = -1;
        for (int b0 = 0; b0 < a.B; b0 += C::NT) {
            int64_t x = 0, own = 0;
            if (b0 + tid < a.B) {
                const Seq s = load_seq<C>(a, plan.side, b0 + tid);
                x = own = (int64_t)a.Hk * s.groups * s.tiles;
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int64_t y = __shfl_up(x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 63) s_part[wave] = x;
            __syncthreads();
            int64_t base = start, sum = 0;
#pragma unroll
            for (int w = 0; w < C::NT / 64; ++w) {
                if (w < wave) base += s_part[w];
                sum += s_part[w];
            }
            const int64_t hi = base + x, lo = hi - own;
            if (own > 0 && lo <= at && at < hi) {
                s_pick = b0 + tid;
                s_pre[0] = lo;
            }
            __syncthreads();
            if (s_pick >= 0) break;
            start += sum;
        }
        b = s_pick;
        start = s_pre[0];
    }

    Worker<C> w(a, lds, s_flag, plan.max_blocks == 1);
    while (at < end) {
        b = __builtin_amdgcn_readfirstlane(b);
        w.b = b;
        w.s = load_seq<C>(a, plan.side, b);
        const int64_t units = (int64_t)a.Hk * w.s.groups;
        while (at < end && at - start < units * w.s.tiles) {
            const int64_t unit = (at - start) / w.s.tiles;
            const int64_t us = start + unit * w.s.tiles, ue = us + w.s.tiles;
            w.h = (int)(unit / w.s.groups);
            const int block = (int)(unit - (int64_t)w.h * w.s.groups) * plan.side + member;
            const int64_t stop = min(end, ue);
            if (block < w.s.blocks) {
                w.begin(block);
                if (!w.s.poison) w.run((int)(at - us), (int)(stop - us));
                w.join_waves();
                const int c0 = (int)(us / share), c1 = (int)((ue - 1) / share);
                bool out = c0 == c1;
                if (!out) {
                    auto slot = [&](int c) {
                        return plan.slots + ((c * plan.side + member) * 2 + (c == c0 ? 1 : 0)) * (int64_t)C::SLOT;
                    };
                    int32_t* arrived = plan.arrived + (c0 * plan.side + member) * C::COUNTERS;
                    const int parts = c1 - c0 + 1, mine = cluster - c0;
                    const int group = C::COUNTERS > 1 ? mine / C::GROUP : 0;
                    const int groups = C::COUNTERS > 1 ? (parts + C::GROUP - 1) / C::GROUP : 1;
                    // Whether this workgroup is the last of n to arrive; where all others have, its
                    // own part stays in registers (KEEP).
                    auto last = [&](int32_t* counter, int n, char* own) {
                        if constexpr (C::KEEP) {
                            if (tid == 0)
                                s_last = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
                            __syncthreads();
                            if (s_last) return true;
                        }
                        w.save(own);
                        __syncthreads();
                        if (tid == 0) s_last = atomicAdd(counter, 1) == n - 1;
                        __syncthreads();
                        return s_last != 0;
                    };
                    // A group's result takes the place of its first part, which has been read by then.
                    int at_level = mine, first = group * C::GROUP, n = min(C::GROUP, parts - first), step = 1;
                    int32_t* counter = arrived + (C::COUNTERS > 1 ? 1 + group : 0);
#pragma unroll 1
                    for (int level = 0;; ++level) {
                        if (!last(counter, n, slot(c0 + at_level))) break;
                        w.join_parts(n, (at_level - first) / step, [&](int i) { return slot(c0 + first + i * step); });
                        if (tid == 0) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                        out = C::COUNTERS == 1 || level == 1 || groups == 1;
                        if (out) break;
                        at_level = first;
                        first = 0;
                        n = groups;
                        step = C::GROUP;
                        counter = arrived;
                        __syncthreads();                 // s_last has been read
                    }
                }
                if (out) w.write(block, w.s.poison);
            }
            at = stop;
        }
        start += units * w.s.tiles;
        ++b;
    }
}

// ------------------------------------------------------------------ host

template <class C>
inline Plan make_plan(int N, int group, bool dense, char* ws) {
    Plan p;
    p.grid = kCUs * C::OCC;
    const int blocks = (N * group + C::BM - 1) / C::BM;
    // Blocks of rows of one (sequence, key head) side by side over the same keys, up to eight,
    // so that they find the keys in L2.  Trees of different sizes would leave members idle:
    // there the blocks follow each other.
    const int rounds = (blocks + 7) / 8;
    p.side = dense ? (blocks + rounds - 1) / rounds : 1;
    p.clusters = p.grid / p.side;
    p.max_blocks = blocks;
    p.arrived = (int32_t*)ws;
    p.slots = ws + kCounterBytes;
    return p;
}

template <class C>
constexpr size_t plan_bytes() {
    return kCounterBytes + (size_t)kCUs * C::OCC * 2 * C::SLOT;
}

template <class C>
inline hipError_t launch_cfg(const AttnArgs& a, hipStream_t stream) {
    const Plan p = make_plan<C>(a.N, a.group, a.offsets == nullptr, a.ws);
    return launch(attn_kernel<C>, dim3((unsigned)p.grid), dim3(C::NT), C::LDS, stream, a, p);
}

// The shape of the tiles by the rows that share keys, N group, and by the units (sequences times key
// heads); f(Cfg) is called with the one that applies.  Few rows: the waves split the keys.  Many rows:
// the waves split the rows and share each tile, the larger the block the fewer the reads of K and V.
// Blocks are no larger than leaves half the CUs one each: then smaller ones join faster (one
// sequence of four key heads, 256 rows each over 2800 keys: 131 us in blocks of 256, 40 us in blocks of
// 64; 32 such sequences, 128 blocks: 93 us in blocks of 256, 98 us in blocks of 128).  17 to 32 rows take the tiles of
// 64 (128 sequences, 32 rows over 2800 keys: 150 us; 165 us with the waves splitting the keys).
template <int IO, int D, class F>
inline auto choose(int rows, int units, F f) {
    if constexpr (IO == GDN_F32) {
        // 256 columns of fp32 for four waves' own keys would not fit the LDS
        if constexpr (D <= 128) {
            if (rows <= 16) return f(Cfg<IO, D, 1, 1, 4, 32, (D <= 64 ? 2 : 1)>{});
        }
        return f(Cfg<IO, D, 1, 4, 1, 32, (D <= 128 ? 2 : 1)>{});
    } else {
        constexpr int occ = D <= 128 ? 2 : 1;
        auto few = [&](int bm) { return (int64_t)units * ((rows + bm - 1) / bm) < kCUs / 2; };
        if (rows <= 16) return f(Cfg<IO, D, 1, 1, 4, 32, occ>{});
        if (rows <= 64 || few(128)) return f(Cfg<IO, D, 2, 2, 2, 32, occ>{});
        if constexpr (D > 128) {
            return f(Cfg<IO, D, 2, 4, 1, 32, 1>{});
        } else {
            if (rows <= 128 || few(256)) return f(Cfg<IO, D, 2, 4, 1, 64, 2>{});
            return f(Cfg<IO, D, 2, 8, 1, 64, 1>{});
        }
    }
}

template <int IO, int D>
inline hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
    return choose<IO, D>(a.N * a.group, a.B * a.Hk, [&](auto c) { return launch_cfg<decltype(c)>(a, stream); });
}
template <int IO, int D>
inline size_t bytes_d(int B, int N, int group, int Hk) {
    return choose<IO, D>(N * group, B * Hk, [](auto c) { return plan_bytes<decltype(c)>(); });
}

}  // namespace attn

// One translation unit each (compiled in parallel).
hipError_t attn_launch_bf16_64(const AttnArgs& a, hipStream_t stream);
hipError_t attn_launch_bf16_128(const AttnArgs& a, hipStream_t stream);
hipError_t attn_launch_bf16_256(const AttnArgs& a, hipStream_t stream);
hipError_t attn_launch_f32_64(const AttnArgs& a, hipStream_t stream);
hipError_t attn_launch_f32_128(const AttnArgs& a, hipStream_t stream);
hipError_t attn_launch_f32_256(const AttnArgs& a, hipStream_t stream);
size_t attn_bytes_bf16_64(int B, int N, int group, int Hk);
size_t attn_bytes_bf16_128(int B, int N, int group, int Hk);
size_t attn_bytes_bf16_256(int B, int N, int group, int Hk);
size_t attn_bytes_f32_64(int B, int N, int group, int Hk);
size_t attn_bytes_f32_128(int B, int N, int group, int Hk);
size_t attn_bytes_f32_256(int B, int N, int group, int Hk);

}  // namespace gdn
