// attn_pages.hip -- the paged cache around the tree attention: append of the
// accepted path's rows, and the pool's bookkeeping (fork, reserve, copy, free,
// compact).
//
// The bookkeeping is integer work on arrays of a few KB to a few MB and bound by the
// latency of its dependent reads.  Where an answer depends on all sequences or all
// pages (which free page a sequence gets, where a page moves) one workgroup does it, so
// that no step waits for another workgroup; what is left (table rows, page copies) is
// spread over the chip.  Counters are changed by integer atomics alone, whose sum
// does not depend on their order.
#include "attn_common.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kOne = 1024;                   // threads of a single-workgroup step
constexpr int kMaxSlots = 4096;
constexpr int kPer = kMaxSlots / kOne;       // slots per thread of such a step

__device__ __forceinline__ bool is_page(int p, int n_pages) { return (uint32_t)p < (uint32_t)n_pages; }

// ------------------------------------------------------------------ append

// Workgroup (b, slice): every slice checks the whole path, so that either all rows of a
// sequence are written or none, then copies its share of the rows: piece e (16 bytes) of
// the pieces of all rows, keys and values.  Bound by the latency of length, path and page id, one
// after the other: 6.1 us for 64 sequences, 5.5 us for one.
template <int ES>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
    __shared__ int s_node[kMaxNodes];
    const int b = blockIdx.x, tid = threadIdx.x;
    const SeqRows rows = seq_rows(a.offsets, b, a.N);
    const int64_t len = a.ctx[b];
    const int want = a.path_len[b];
    const int n = max(rows.n, 0);
    const int first = (int)(len / (int64_t)a.page.d);
    bool bad = len < 0 || want > n;
    const int m = bad ? 0 : max(want, 0);
    if (m > 0) {
        const int64_t last = (len + m - 1) / (int64_t)a.page.d;
        bad |= last >= a.width || len + m > 0x7fffffff;      // new_len has 31 bits
        if (!bad) {
            for (int t = tid; t < m; t += kThreads) {
                const int i = a.path[rows.row0 + t];
                s_node[t] = i;
                bad |= i < 0 || i >= n;
            }
            for (int c = first + tid; c <= (int)last; c += kThreads)
                bad |= !is_page(a.table[(int64_t)b * a.width + c], a.n_pages);
        }
    }
    bad = __syncthreads_or(bad) != 0;
    if (blockIdx.y == 0 && tid == 0) a.new_len[b] = bad ? -1 : (int32_t)(len + m);
    if (bad || m == 0) return;
    constexpr int E = 16 / ES;
    const int per_head = a.d / E, per_row = per_head * a.Hk;
    const int pieces = 2 * m * per_row;
    for (int e = blockIdx.y * kThreads + tid; e < pieces; e += gridDim.y * kThreads) {
        const int kv = e & 1;
        const int x = e >> 1;
        const int t = x / per_row, y = x - t * per_row;
        const int h = y / per_head, c = y - h * per_head;
        const int64_t at = len + t;
        const int64_t col = at / (int64_t)a.page.d;
        const int64_t pid = a.table[(int64_t)b * a.width + col];
        const Rows& in = kv ? a.v : a.k;
        const Pool& out = kv ? a.vp : a.kp;
        const char* src = in.p + ((rows.row0 + s_node[t]) * in.row + h * in.head + c * E) * ES;
        char* dst = out.p + (pid * out.page + (at - col * a.page.d) * out.row + h * out.head + c * E) * ES;
        *(uint4*)dst = *(const uint4*)src;
    }
}

// ------------------------------------------------------------------ copy

// Pages that are one dense run of bytes in memory (rows first or heads first), 4 KB to a workgroup,
// one 16-byte piece to a thread; pool by pool and layer by layer, so that all that runs at a time
// lies in one of them.  Bound by memory (2500 pages of 4 layers, 32 KB each: 3.6 TB/s read and
// written; longer loops per workgroup and pages outermost were slower, 468 us for 369, and stores
// that the L2 keeps 405).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kCopyGrid = 1 << 20;
template <int ES>
__global__ __launch_bounds__(kThreads) void copy_dense_kernel(CopyArgs a, FastDiv chunks, int bytes) {
    const uint32_t n = (uint32_t)max(min(*a.count, a.n), 0);
    const uint32_t run = n * chunks.d, total = run * 2 * (uint32_t)a.n_layers;
    for (uint32_t w = blockIdx.x; w < total; w += gridDim.x) {
        const uint32_t part = w / run, y = w - part * run;
        const uint32_t i = quot(chunks, y), chunk = y - i * chunks.d;
        const int s = a.src[i], t = a.dst[i];
        const int at = ((int)chunk * kThreads + (int)threadIdx.x) * 16;
        if (!is_page(s, a.n_pages) || !is_page(t, a.n_pages) || at >= bytes) continue;
        const int64_t layer = part >> 1;
        const Pool& pool = part & 1 ? a.vp : a.kp;
        char* base = pool.p + layer * (part & 1 ? a.v_layer : a.k_layer) * ES + at;
        const u32x4 x = *(const u32x4*)(base + s * pool.page * ES);
        __builtin_nontemporal_store(x, (u32x4*)(base + t * pool.page * ES));
    }
}

// Any strides: a workgroup copies one page of one layer's keys or values.
template <int ES>
__global__ __launch_bounds__(kThreads) void copy_strided_kernel(CopyArgs a) {
    const int n = min(*a.count, a.n);
    const int64_t total = (int64_t)n * a.n_layers * 2;
    constexpr int E = 16 / ES;
    const int per_head = a.d / E, pieces = per_head * a.Hk * a.page_rows;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int kv = (int)(w & 1);
        const int layer = (int)((w >> 1) % a.n_layers), i = (int)((w >> 1) / a.n_layers);
        const int s = a.src[i], t = a.dst[i];
        if (!is_page(s, a.n_pages) || !is_page(t, a.n_pages)) continue;
        const Pool& pool = kv ? a.vp : a.kp;
        char* base = pool.p + (int64_t)layer * (kv ? a.v_layer : a.k_layer) * ES;
        for (int e = threadIdx.x; e < pieces; e += kThreads) {
            const int c = e % per_head, y = e / per_head;
            const int64_t in_page = (int64_t)(y / a.Hk) * pool.row + (int64_t)(y % a.Hk) * pool.head + c * E;
            *(uint4*)(base + (t * pool.page + in_page) * ES) = *(const uint4*)(base + (s * pool.page + in_page) * ES);
        }
    }
}

// ------------------------------------------------------------------ fork, free

__global__ __launch_bounds__(kThreads) void fork_kernel(PageArgs a, int n, const int32_t* src_seq,
                                                       const int32_t* dst_seq, int32_t* status) {
    const int i = blockIdx.x, tid = threadIdx.x;
    const int s = src_seq[i], t = dst_seq[i];
    bool bad = (uint32_t)s >= (uint32_t)a.n_slots || (uint32_t)t >= (uint32_t)a.n_slots;
    for (int j = tid; j < n; j += kThreads) bad |= dst_seq[j] == s || (j < i && dst_seq[j] == t);
    int64_t used = 0;
    int len = 0;
    if (!bad) {
        len = a.length[s];
        used = ((int64_t)len + a.page_rows - 1) / a.page_rows;
        bad = len < 0 || used > a.held[s] || used > a.width || a.held[t] != 0;
        if (!bad)
            for (int c = tid; c < used; c += kThreads) bad |= !is_page(a.table[(int64_t)s * a.width + c], a.n_pages);
    }
    bad = __syncthreads_or(bad) != 0;
    if (tid == 0) status[i] = bad ? -1 : 0;
    if (bad) return;
    for (int c = tid; c < a.width; c += kThreads) {
        int p = -1;
        if (c < used) {
            p = a.table[(int64_t)s * a.width + c];
            atomicAdd(&a.ref[p], 1);
        }
        a.table[(int64_t)t * a.width + c] = p;
    }
    if (tid == 0) {
        a.held[t] = (int)used;
        a.length[t] = len;
    }
}

__global__ __launch_bounds__(kThreads) void free_kernel(PageArgs a, const int32_t* drop) {
    const int s = blockIdx.x, tid = threadIdx.x;
    if (drop[s] == 0) return;
    const int held = min(a.held[s], a.width);
    for (int c = tid; c < a.width; c += kThreads) {
        int32_t* e = &a.table[(int64_t)s * a.width + c];
        if (c < held && is_page(*e, a.n_pages)) atomicSub(&a.ref[*e], 1);
        *e = -1;
    }
    __syncthreads();                         // every thread has read held
    if (tid == 0) {
        a.held[s] = 0;
        a.length[s] = 0;
    }
}

// ------------------------------------------------------------------ reserve, compact

// Exclusive sum over the kOne threads of a workgroup; `part` holds kOne / 64 words.  Two
// barriers.
template <class T>
__device__ __forceinline__ T block_exclusive(T x, T* part, T& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T run = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T y = __shfl_up(run, o);
        if (lane >= o) run += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = run;
    __syncthreads();
    T base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kOne / 64; ++w) {
        if (w < wave) base += part[w];
        total += part[w];
    }
    return base + run - x;
}

// kScan consecutive pages per thread and round.
constexpr int kScan = 8;
__device__ __forceinline__ uint32_t scan_pages(const int32_t* ref, int p0, int n_pages, bool free_ones) {
    uint32_t bits = 0;
    if (p0 + kScan <= n_pages) {
        int r[kScan];
#pragma unroll
        for (int i = 0; i < kScan; i += 4) {
            const int4 q = *(const int4*)(ref + p0 + i);
            r[i] = q.x; r[i + 1] = q.y; r[i + 2] = q.z; r[i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < kScan; ++i) bits |= ((r[i] > 0) != free_ones ? 1u : 0u) << i;
    } else {
        for (int i = 0; i < kScan && p0 + i < n_pages; ++i)
            bits |= ((ref[p0 + i] > 0) != free_ones ? 1u : 0u) << i;
    }
    return bits;
}

// The free page with rank f goes to the sequence s with first[s] <= f < first[s + 1].  A shared
// last page is counted in a hash table in LDS (page, sequences that ask, the last of them).  160
// slots over 6000 pages: 15.8 us, the chain of these reads, sums and barriers (23.6 us where each
// thread hands out the free pages that it found).
__global__ __launch_bounds__(kOne) void reserve_kernel(PageArgs a, const int32_t* need, int32_t* src, int32_t* dst,
                                                      int32_t* count, int32_t* status, int buckets) {
    __shared__ int64_t s_first[kMaxSlots + 1];
    __shared__ int64_t s_part[kOne / 64];
    __shared__ int s_cpart[kOne / 64];
    __shared__ uint16_t s_free[kOne * kScan];
    extern __shared__ int s_hash[];          // key, askers, last asker: buckets each
    int* key = s_hash;
    int* askers = s_hash + buckets;
    int* last = s_hash + 2 * buckets;
    const int tid = threadIdx.x, S = a.n_slots;
    for (int i = tid; i < buckets; i += kOne) {
        key[i] = -1;
        askers[i] = 0;
        last[i] = -1;
    }
    __syncthreads();
    // 1. what each sequence asks for; thread t has slots t kPer .. t kPer + kPer - 1
    int len[kPer], held[kPer], tail[kPer], bucket[kPer], refs[kPer];
    int64_t want[kPer];
    bool wants[kPer], fits[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = tid * kPer + u;
        wants[u] = fits[u] = false;
        bucket[u] = -1;
        tail[u] = refs[u] = len[u] = held[u] = 0;
        want[u] = 0;
        if (s >= S) continue;
        const int more = need[s];
        len[u] = a.length[s];
        held[u] = a.held[s];
        wants[u] = more > 0;
        want[u] = ((int64_t)len[u] + more + a.page_rows - 1) / a.page_rows;
        fits[u] = wants[u] && len[u] >= 0 && held[u] >= 0 && want[u] <= a.width && held[u] <= a.width &&
                  len[u] <= (int64_t)held[u] * a.page_rows;
        if (fits[u] && len[u] % a.page_rows > 0) {
            tail[u] = a.table[(int64_t)s * a.width + len[u] / a.page_rows];
            fits[u] = is_page(tail[u], a.n_pages);
            if (fits[u]) refs[u] = a.ref[tail[u]];
        }
        if (refs[u] > 1) {
            uint32_t at = ((uint32_t)tail[u] * 2654435761u) & (uint32_t)(buckets - 1);
            for (;;) {                       // twice as many buckets as slots: one is free
                const int old = atomicCAS(&key[at], -1, tail[u]);
                if (old == -1 || old == tail[u]) break;
                at = (at + 1) & (uint32_t)(buckets - 1);
            }
            bucket[u] = (int)at;
            atomicAdd(&askers[at], 1);
            atomicMax(&last[at], s);
        }
    }
    __syncthreads();
    int64_t demand[kPer], mine = 0;
    bool copies[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = tid * kPer + u;
        copies[u] = bucket[u] >= 0 && !(askers[max(bucket[u], 0)] == refs[u] && last[max(bucket[u], 0)] == s);
        demand[u] = fits[u] ? max(want[u] - held[u], (int64_t)0) + copies[u] : 0;
        mine += demand[u];
    }
    int64_t asked;
    int64_t run = block_exclusive<int64_t>(mine, s_part, asked);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        s_first[tid * kPer + u] = run;
        run += demand[u];
    }
    if (tid == kOne - 1) s_first[kMaxSlots] = run;
    // 2. free pages, counted until they are enough
    int64_t free_pages = 0;
    for (int p0 = 0; p0 < a.n_pages && free_pages < asked; p0 += kOne * kScan) {
        int total;
        block_exclusive<int>(__popc(scan_pages(a.ref, p0 + tid * kScan, a.n_pages, true)), s_cpart, total);
        free_pages += total;
    }
    // 3. who is served.  Ranks only grow, so the served ones are those whose last rank is in reach.
    int ncopy = 0;
    int64_t top = 0;
    bool good[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = tid * kPer + u;
        const int64_t upto = s_first[s] + demand[u];
        good[u] = fits[u] && (upto <= free_pages || (demand[u] == 0 && bucket[u] < 0));
        copies[u] = copies[u] && good[u];
        ncopy += copies[u];
        if (good[u] && demand[u] > 0) top = max(top, upto);
        if (s < S) status[s] = !wants[u] || good[u] ? 0 : fits[u] ? -2 : -1;
    }
    int total_copies;
    int at_copy = block_exclusive<int>(ncopy, s_cpart, total_copies);
    if (tid == 0) *count = total_copies;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, (int64_t)__shfl_xor(top, o));
    __syncthreads();
    if ((tid & 63) == 0) s_part[tid >> 6] = top;
    // the hash table is done with: per slot, where its copy goes in the list (or -1), the column of
    // its last page and that of its first missing one
    int* copy_at = s_hash;
    int* tail_col = s_hash + S;
    int* next_col = s_hash + 2 * S;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int s = tid * kPer + u;
        if (s >= S) continue;
        copy_at[s] = copies[u] ? at_copy++ : -1;
        tail_col[s] = len[u] / a.page_rows;
        next_col[s] = held[u];
        if (good[u]) a.held[s] = max((int)want[u], held[u]);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kOne / 64; ++w) top = max(top, s_part[w]);
    // 4. hand the pages out: the free ones of a round are listed by rank, a thread takes a rank
    int64_t base = 0;
    for (int p0 = 0; p0 < a.n_pages && base < top; p0 += kOne * kScan) {
        uint32_t bits = scan_pages(a.ref, p0 + tid * kScan, a.n_pages, true);
        int total;
        int at = block_exclusive<int>(__popc(bits), s_cpart, total);
        for (; bits; bits &= bits - 1) s_free[at++] = (uint16_t)(tid * kScan + __ffs(bits) - 1);
        __syncthreads();
        const int take = (int)min((int64_t)total, top - base);
        for (int x = tid; x < take; x += kOne) {
            const int p = p0 + s_free[x];
            const int64_t f = base + x;
            int lo = 0, hi = S;              // first[lo] <= f < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] <= f) lo = mid; else hi = mid;
            }
            const int s = lo;
            const int off = (int)(f - s_first[s]);
            const int c = copy_at[s];
            a.ref[p] = 1;
            if (c >= 0 && off == 0) {
                int32_t* e = &a.table[(int64_t)s * a.width + tail_col[s]];
                const int old = *e;
                src[c] = old;
                dst[c] = p;
                atomicSub(&a.ref[old], 1);
                *e = p;
            } else {
                a.table[(int64_t)s * a.width + next_col[s] + off - (c >= 0 ? 1 : 0)] = p;
            }
        }
        base += total;
    }
}

// 18 000 pages: 22 us, two passes over the counts in rounds of 8192 pages and the moves.
__global__ __launch_bounds__(kOne) void compact_kernel(PageArgs a, int n, int32_t* src, int32_t* dst,
                                                      int32_t* count, int32_t* remap) {
    __shared__ int s_part[kOne / 64];
    const int tid = threadIdx.x;
    int held = 0;                            // pages held: the new front
    for (int p0 = 0; p0 < a.n_pages; p0 += kOne * kScan) {
        int total;
        block_exclusive<int>(__popc(scan_pages(a.ref, p0 + tid * kScan, a.n_pages, false)), s_part, total);
        held += total;
    }
    // ranks of the free pages below `held` and of the held ones from there on
    int holes = 0, moves = 0;
    for (int p0 = 0; p0 < a.n_pages; p0 += kOne * kScan) {
        const int p = p0 + tid * kScan;
        const int here = min(max(a.n_pages - p, 0), kScan);
        const int below = min(max(held - p, 0), here);
        const uint32_t live = scan_pages(a.ref, p, a.n_pages, false);
        const uint32_t low = (1u << below) - 1u;
        uint32_t hole = ~live & low, move = live & ~low;
        int th, tm;
        int rh = holes + block_exclusive<int>(__popc(hole), s_part, th);
        int rm = moves + block_exclusive<int>(__popc(move), s_part, tm);
        for (int i = 0; i < here; ++i) {
            if ((hole >> i) & 1u) {
                if (rh < n) dst[rh] = p + i;
                ++rh;
            }
            if ((move >> i) & 1u) {
                if (rm < n) src[rm] = p + i;
                ++rm;
            }
            remap[p + i] = p + i;
        }
        holes += th;
        moves += tm;
    }
    const int m = min(moves, n);             // as many holes as moves
    if (tid == 0) *count = m;
    __syncthreads();
    for (int i = tid; i < m; i += kOne) {
        const int s = src[i], t = dst[i];
        remap[s] = t;
        a.ref[t] = a.ref[s];
        a.ref[s] = 0;
    }
}

__global__ __launch_bounds__(kThreads) void remap_kernel(PageArgs a, const int32_t* remap) {
    const int64_t total = (int64_t)a.n_slots * a.width;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int p = a.table[i];
        if (is_page(p, a.n_pages)) {
            const int q = remap[p];
            if (q != p) a.table[i] = q;
        }
    }
}

// Whether a page's elements fill page_rows h_kv d consecutive ones, rows first or heads first.
bool dense(const Pool& p, int rows, int h, int d) {
    const bool rows_first = (h == 1 || p.head == d) && (rows == 1 || p.row == (int64_t)h * d);
    const bool heads_first = (rows == 1 || p.row == d) && (h == 1 || p.head == (int64_t)rows * d);
    return rows_first || heads_first;
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int io, hipStream_t stream) {
    const int es = io == GDN_F32 ? 4 : 2;
    // Workgroups per sequence: one for each 32 KiB that a path of every eighth node takes, the
    // length of the paths that trees are accepted by; a longer path loops.
    const int64_t bytes = (int64_t)((a.N + 7) / 8) * a.Hk * a.d * es * 2;
    const unsigned slices = (unsigned)std::min<int64_t>(16, (bytes + 32767) / 32768);
    return launch(es == 4 ? append_kernel<4> : append_kernel<2>, dim3((unsigned)a.B, slices), dim3(kThreads), 0,
                  stream, a);
}

hipError_t launch_pages_copy(const CopyArgs& a, int io, hipStream_t stream) {
    const int es = io == GDN_F32 ? 4 : 2;
    const int64_t parts = (int64_t)a.n * a.n_layers * 2;
    const int64_t bytes = (int64_t)a.page_rows * a.Hk * a.d * es, chunks = (bytes + kThreads * 16 - 1) / (kThreads * 16);
    if (dense(a.kp, a.page_rows, a.Hk, a.d) && dense(a.vp, a.page_rows, a.Hk, a.d) && bytes < (1 << 30) &&
        parts * chunks + kCopyGrid < 0xffffffffLL && (int64_t)a.n * chunks < (1LL << 31)) {
        const unsigned grid = (unsigned)std::min<int64_t>(parts * chunks, kCopyGrid);
        return launch(es == 4 ? copy_dense_kernel<4> : copy_dense_kernel<2>, dim3(grid), dim3(kThreads), 0, stream, a,
                      fast_div((uint32_t)chunks), (int)bytes);
    }
    const unsigned grid = (unsigned)std::min<int64_t>(parts, 256 * 8);
    return launch(es == 4 ? copy_strided_kernel<4> : copy_strided_kernel<2>, dim3(grid), dim3(kThreads), 0, stream, a);
}

hipError_t launch_pages_fork(const PageArgs& a, int n, const int32_t* src_seq, const int32_t* dst_seq,
                             int32_t* status, hipStream_t stream) {
    return launch(fork_kernel, dim3((unsigned)n), dim3(kThreads), 0, stream, a, n, src_seq, dst_seq, status);
}

hipError_t launch_pages_reserve(const PageArgs& a, const int32_t* need, int32_t* src, int32_t* dst,
                                int32_t* count, int32_t* status, hipStream_t stream) {
    int buckets = 64;
    while (buckets < 2 * a.n_slots) buckets *= 2;
    return launch(reserve_kernel, dim3(1), dim3(kOne), (size_t)buckets * 12, stream, a, need, src, dst, count,
                  status, buckets);
}

hipError_t launch_pages_free(const PageArgs& a, const int32_t* drop, hipStream_t stream) {
    return launch(free_kernel, dim3((unsigned)a.n_slots), dim3(kThreads), 0, stream, a, drop);
}

hipError_t launch_pages_compact(const PageArgs& a, int n, int32_t* src, int32_t* dst, int32_t* count,
                                int32_t* remap, hipStream_t stream) {
    hipError_t e = launch(compact_kernel, dim3(1), dim3(kOne), 0, stream, a, n, src, dst, count, remap);
    if (e != hipSuccess) return e;
    const int64_t total = (int64_t)a.n_slots * a.width;
    const unsigned grid = (unsigned)std::min<int64_t>((total + kThreads - 1) / kThreads, 256 * 8);
    return launch(remap_kernel, dim3(grid), dim3(kThreads), 0, stream, a, (const int32_t*)remap);
}

}  // namespace gdn
