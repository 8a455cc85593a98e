// paged_cache.cu -- the upkeep of a paged key-value cache: writing new tokens, growing and
// shrinking sequences with copy on write, sharing pages with a new sequence, compaction.
//
// Which pages are free is ref[p] == 0, nothing else: no free list to keep in step.  A call that
// takes pages takes the lowest free ones, row after row, so the outcome depends on the inputs
// alone.  Finding them is a ranking of the free pages (how many free pages lie below p), which a
// cluster of 8 or 16 blocks does in one launch: ref is cut into up to MAXCH chunks, warps count the
// free pages of theirs and leave the counts in every block's shared memory (distributed shared
// memory), each block sums them up, and the chunks that hold pages to hand out are dealt over the
// cluster's warps once more.  What is to be done to keys, values and tables follows in a second
// kernel over the whole GPU, launched as a dependent of the first, whose end it waits for on the
// device.
#include <limits.h>

#include <cooperative_groups.h>

#include "common.cuh"
#include "paged.cuh"

namespace gret {

namespace cg = cooperative_groups;

namespace {

constexpr int CL_FEW = 8;              // blocks of a planning cluster: the portable maximum,
constexpr int CL_MANY = 16;            // and what the GPU allows, for pools of
constexpr int MANY_PAGES = 1 << 17;    // so many pages (131072 of them, 1000 rows that come and go:
                                       // 21.3 -> 18.7 us; 30000 to 110000 pages 1 to 2 % slower)
constexpr int PNT = 1024;
constexpr int PNW = PNT / 32;
constexpr int MAXCH = 4 * PNT;         // chunks of ref
constexpr int GROUP = 4;               // chunks a warp counts at once
constexpr int GRID = 148 * 4;          // blocks of the kernels that carry a plan out
constexpr int NT = 256;
constexpr int APPLY_SM = 6;            // of a resize's an SM: its rows wait for lists and counts
constexpr int64_t FORK_ALONE = 1 << 21;   // pairs x table entries that one fork kernel does

// Exclusive sums of x and y over the block's threads, and the totals.  `sums` has 2 PNW entries.
struct Sums {
    int64_t x, all_x;
    int y, all_y;
};

__device__ __forceinline__ Sums block_scan(int64_t x, int y, int64_t (*sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t ix = x;
    int iy = y;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x2 = __shfl_up_sync(0xffffffffu, ix, o);
        const int y2 = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += x2;
            iy += y2;
        }
    }
    if (lane == 31) {
        sums[warp][0] = ix;
        sums[warp][1] = iy;
    }
    __syncthreads();
    int64_t wx = sums[lane][0];              // PNW = 32: every warp scans the warps' sums
    int wy = (int)sums[lane][1];
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x2 = __shfl_up_sync(0xffffffffu, wx, o);
        const int y2 = __shfl_up_sync(0xffffffffu, wy, o);
        if (lane >= o) {
            wx += x2;
            wy += y2;
        }
    }
    Sums r;
    r.all_x = __shfl_sync(0xffffffffu, wx, 31);
    r.all_y = __shfl_sync(0xffffffffu, wy, 31);
    const int64_t bx = __shfl_sync(0xffffffffu, wx, warp ? warp - 1 : 0);
    const int by = __shfl_sync(0xffffffffu, wy, warp ? warp - 1 : 0);
    r.x = (warp ? bx : 0) + ix - x;
    r.y = (warp ? by : 0) + iy - y;
    return r;
}

// ref, read 16 bytes at a time whatever its alignment: quad j is the entries 4 j - skew and on,
// where entries before the first and from P on count as taken.  Chunk c is the quads [c * step, c *
// step + step).
struct Chunks {
    const int32_t* ref;
    int P, skew, step, n;

    __device__ __forceinline__ Chunks(const int32_t* r, int pages)
        : ref(r), P(pages), skew((int)(reinterpret_cast<uintptr_t>(r) >> 2 & 3)) {
        const int quads = (int)(((int64_t)P + skew + 3) / 4);
        step = ((quads + MAXCH - 1) / MAXCH + 31) / 32 * 32;
        n = (quads + step - 1) / step;
    }
    __device__ __forceinline__ int entry(int quad) const { return 4 * quad - skew; }
    __device__ __forceinline__ bool inside(int quad) const {
        return entry(quad) >= 0 && entry(quad) + 4 <= P;
    }
    __device__ __forceinline__ int4 inner_quad(int quad) const {
        return *reinterpret_cast<const int4*>(ref + entry(quad));
    }
    __device__ __forceinline__ int4 quad(int q) const {
        if (inside(q)) return inner_quad(q);
        int x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = entry(q) + e >= 0 && entry(q) + e < P ? ref[entry(q) + e] : 1;
        return make_int4(x[0], x[1], x[2], x[3]);
    }
};

__device__ __forceinline__ int free_of(int4 q) {
    return (q.x == 0) + (q.y == 0) + (q.z == 0) + (q.w == 0);
}

// The four entries' ranks among the free pages, `before` of which lie before the warp's quads and,
// afterwards, before the next ones.
__device__ __forceinline__ int4 ranks_of(int4 q, int& before) {
    const int lane = threadIdx.x & 31, mine = free_of(q);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    int4 r;
    r.x = before + incl - mine;
    r.y = r.x + (q.x == 0);
    r.z = r.y + (q.y == 0);
    r.w = r.z + (q.z == 0);
    before += __shfl_sync(0xffffffffu, incl, 31);
    return r;
}

// Counts each chunk's free pages into `count` [MAXCH] of every block of the cluster.  Starts with
// the second half of a cluster barrier (whoever calls has arrived) and ends with a whole one: what
// the cluster's blocks read of the inputs beforehand, no block changes before that.
template <int CL>
__device__ __forceinline__ void count_free(const Chunks& ch, int* count) {
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = cluster.block_rank() * PNW + (threadIdx.x >> 5);
    bool begun = false;
    for (int c0 = warp; c0 < ch.n; c0 += CL * PNW * GROUP) {
        int n[GROUP] = {};
        bool whole[GROUP];                       // chunks that lie in ref with all their quads
#pragma unroll
        for (int g = 0; g < GROUP; ++g) {
            const int c = c0 + g * CL * PNW;
            whole[g] = c < ch.n && ch.inside(c * ch.step) && ch.inside((c + 1) * ch.step - 1);
        }
        // all loads of an iteration are on their way before the first is looked at
#pragma unroll 2
        for (int i = lane; i < ch.step; i += 32) {
            int4 x[GROUP];
#pragma unroll
            for (int g = 0; g < GROUP; ++g) {
                x[g] = make_int4(1, 1, 1, 1);
                if (whole[g]) x[g] = ch.inner_quad((c0 + g * CL * PNW) * ch.step + i);
            }
#pragma unroll
            for (int g = 0; g < GROUP; ++g) n[g] += free_of(x[g]);
        }
#pragma unroll
        for (int g = 0; g < GROUP; ++g) {
            const int c = c0 + g * CL * PNW;
            if (c < ch.n && !whole[g])
                for (int i = lane; i < ch.step; i += 32) n[g] += free_of(ch.quad(c * ch.step + i));
        }
        if (!begun) cluster.barrier_wait();      // every block runs: its shared memory is there
        begun = true;
#pragma unroll
        for (int g = 0; g < GROUP; ++g) {
            const int c = c0 + g * CL * PNW;
            const int sum = __reduce_add_sync(0xffffffffu, n[g]);
            if (c < ch.n && lane < CL) cluster.map_shared_rank(count, lane)[c] = sum;
        }
    }
    if (!begun) cluster.barrier_wait();
    cluster.sync();
}

// Turns the counts into the free pages before each chunk, and returns all of them; the exclusive
// sum of x over the block's threads goes along.
__device__ __forceinline__ int rank_free(const Chunks& ch, int* count, int64_t (*sums)[2],
                                         int64_t& x) {
    constexpr int PER = MAXCH / PNT;
    int n[PER], mine = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int c = threadIdx.x * PER + k;
        n[k] = c < ch.n ? count[c] : 0;
        mine += n[k];
    }
    const Sums r = block_scan(x, mine, sums);
    x = r.x;
    int run = r.y;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        count[threadIdx.x * PER + k] = run;
        run += n[k];
    }
    return r.all_y;
}

// Division by a number known on the host, for dividends below 2^31, by multiplication (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994): with s = ceil(log2 d)
// and m = floor(2^32 (2^s - d) / d) + 1, n / d = (floor(m n / 2^32) + n) >> s.
struct FastDiv {
    uint32_t d, m;
    int s;

    explicit FastDiv(uint32_t x) : d(x), s(0) {
        while ((1u << s) < d) ++s;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

// A page as 16-byte pieces, in the order of its addresses: heads inside tokens, or tokens inside
// heads where heads lie further apart.
struct Pieces {
    FastDiv outer, row;          // pieces an outer step, pieces a row
    int64_t so, si;              // bytes an outer step, an inner one
    int total;                   // pieces a page
    bool tokens_inside;

    explicit Pieces(const PagedPool& p)
        : outer((uint32_t)((p.sh > p.st ? 1 << p.page_shift : p.H) * (p.row_bytes / 16))),
          row((uint32_t)(p.row_bytes / 16)),
          so(p.sh > p.st ? p.sh : p.st),
          si(p.sh > p.st ? p.st : p.sh),
          total((int)(p.H * (p.row_bytes / 16) << p.page_shift)),
          tokens_inside(p.sh > p.st) {}
};

// The pieces [c0, c0 + NT) of the slots below `slots` of page `from`, to page `to`, by a block.  One
// piece of keys and one of values a thread: four blocks an SM then have 32 KB on their way, enough
// to hide HBM's latency; with 64 or 128 KB reads and writes get in each other's way (16448 moves of
// 64 KB: 330, 351 and 360 us).
__device__ __forceinline__ void copy_pieces(const PagedPool& p, const Pieces& pc, int64_t from,
                                            int64_t to, int c0, int slots) {
    const uint32_t c = c0 + threadIdx.x;
    const uint32_t o = pc.outer.div(c), r = c - o * pc.outer.d, i = pc.row.div(r);
    if (c < (uint32_t)pc.total && (int)(pc.tokens_inside ? i : o) < slots) {
        const int64_t off = o * pc.so + i * pc.si + (r - i * pc.row.d) * 16;
        const uint4 k = *reinterpret_cast<const uint4*>(p.k + from * p.sp + off);
        const uint4 v = *reinterpret_cast<const uint4*>(p.v + from * p.sp + off);
        *reinterpret_cast<uint4*>(p.k + to * p.sp + off) = k;
        *reinterpret_cast<uint4*>(p.v + to * p.sp + off) = v;
    }
}

// Whether the current device places clusters of CL_MANY blocks of a planning kernel with up to `smem`
// bytes, asked once on each of the first 64 devices.
template <auto Kernel>
bool many_blocks(int smem) {
    static std::atomic<uint64_t> asked{0}, fits{0};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device >= 64) return false;
    const uint64_t bit = (uint64_t)1 << device;
    if (!(asked.load(std::memory_order_acquire) & bit)) {
        cudaLaunchAttribute dims;
        dims.id = cudaLaunchAttributeClusterDimension;
        dims.val.clusterDim.x = CL_MANY;
        dims.val.clusterDim.y = dims.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(CL_MANY);
        cfg.blockDim = dim3(PNT);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &dims;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok =
            cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                cudaSuccess &&
            cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
                cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) == cudaSuccess && n > 0;
        cudaGetLastError();      // an answer of no leaves no error behind
        if (ok) fits.fetch_or(bit, std::memory_order_release);
        asked.fetch_or(bit, std::memory_order_release);
    }
    return fits.load(std::memory_order_acquire) & bit;
}

// ---------------------------------------------------------------------------------------------
// append: a copy of every token's row of heads to its slot.  Bound by HBM, each byte read and
// written once; with few tokens by the chain row -> position -> page -> copy, so a warp's lanes find
// the places of its tokens side by side, and a warp takes several only when there are more tokens
// than warps to go round.  Measured, 8 heads of 128 in bf16: 176,600 tokens 228 us (6.3 TB/s), 256
// single tokens 2.6 us.

constexpr int AP_MAXTOK = 8;           // tokens of one warp
constexpr int AP_U = 4;                // pieces of keys, and of values, in flight a lane

// The last of S rows that begins at or before token i (the first, if none does).
__device__ __forceinline__ int row_of(const int32_t* cu, int S, int64_t i) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = S;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool below = lane * step < n && (lane == 0 || cu[lo + lane * step] <= i);
        const int last = __popc(__ballot_sync(0xffffffffu, below)) - 1;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__global__ void __launch_bounds__(NT) append_kernel(const PagedAppendArgs a, const FastDiv token,
                                                    const FastDiv row, const int tok) {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t i0 = ((int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5)) * tok;
    if (i0 >= a.T) return;
    const int64_t i = i0 + lane;                  // this lane's token
    int64_t slot = -1;
    int b = a.cu_seqlens ? row_of(a.cu_seqlens, a.table.S, i0) : (int)i;
    if (lane < tok && i < a.T) {
        int64_t at = 0;
        bool in = true;
        if (a.cu_seqlens) {
            while (b < a.table.S && a.cu_seqlens[b + 1] <= i) ++b;
            in = b < a.table.S && i >= a.cu_seqlens[b];     // not around the sequences
            if (in) at = i - a.cu_seqlens[b];
        }
        const int pos = in ? a.pos[b] : -1;
        if (pos >= 0) {
            at += pos;
            if (at >= (int64_t)a.table.max_pages << a.pool.page_shift) {
                paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            } else {
                const int id = a.table.entries[b * a.table.stride + (at >> a.pool.page_shift)];
                if ((unsigned)id >= (unsigned)a.pool.n_pages)
                    paged_flag(a.status, GRET_PAGED_BAD_PAGE);
                else
                    slot = id * a.pool.sp + (at & ((1 << a.pool.page_shift) - 1)) * a.pool.st;
            }
        }
    }
    const uint32_t total = min((int64_t)tok, a.T - i0) * token.d;
    for (uint32_t c0 = 0; c0 < total; c0 += 32 * AP_U) {
        uint4 k[AP_U], v[AP_U];
        int64_t to[AP_U];
#pragma unroll
        for (int u = 0; u < AP_U; ++u) {
            const uint32_t c = c0 + u * 32 + lane;
            const uint32_t t = token.div(c), r = c - t * token.d, h = row.div(r);
            const uint32_t x = (r - h * row.d) * 16;
            to[u] = __shfl_sync(0xffffffffu, slot, t & 31);
            if (c >= total) to[u] = -1;
            if (to[u] >= 0) {
                to[u] += h * a.pool.sh + x;
                k[u] = *reinterpret_cast<const uint4*>(a.k + (i0 + t) * a.kt + h * a.kh + x);
                v[u] = *reinterpret_cast<const uint4*>(a.v + (i0 + t) * a.vt + h * a.vh + x);
            }
        }
#pragma unroll
        for (int u = 0; u < AP_U; ++u)
            if (to[u] >= 0) {
                *reinterpret_cast<uint4*>(a.pool.k + to[u]) = k[u];
                *reinterpret_cast<uint4*>(a.pool.v + to[u]) = v[u];
            }
    }
}

// ---------------------------------------------------------------------------------------------
// resize: a plan by one cluster (who gets which page), then the whole GPU carries it out.  Latency
// bounds it: of a step of 256 rows on 20000 pages (9.7 us) the plan takes 7 (rows 1.5, counting 1.4,
// the cluster's barrier and the sums 1.2, handing out 1.5, the launch the rest) and the copies 2.7;
// of 1000 rows that come and go on 786433 pages (24 us) counting takes 5.5 (it reads 0.8 TB/s, with
// 8 blocks or 16: they share one GPC's way to the L2), handing out 6, and the rows' lists 4.

// A row's change, from its length before the call.
struct Change {
    int64_t n0, n1;
    bool bad;            // the length is none that the table can hold
};

__device__ __forceinline__ Change change_of(const PagedResizeArgs& a, int s) {
    Change c;
    c.n0 = a.seq_lens[s];
    c.n1 = c.n0 + a.delta[s];
    if (c.n1 < 0) c.n1 = 0;
    c.bad = c.n0 < 0 || c.n0 > (int64_t)a.table.max_pages << a.pool.page_shift;
    return c;
}

// What the rows [s0, s1) ask for: pages in all, each row's to upto, the table entry that the first goes
// to, and where `lead` the plan in workspace and pos.
template <int U>
__device__ __forceinline__ int64_t needs_of(const PagedResizeArgs& a, int s0, int s1, bool lead,
                                            int* upto, int* first) {
    const int shift = a.pool.page_shift;
    int64_t mine = 0;
    for (int sb = s0; sb < s1; sb += U) {
        // length, last page, its count: three loads one after another, of U rows side by side
        Change c[U];
        int id[U], count[U];
        bool fits[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u] = {0, 0, false};
            if (sb + u < s1) c[u] = change_of(a, sb + u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool grows = !c[u].bad && c[u].n1 > c[u].n0;
            fits[u] = grows && c[u].n1 <= (int64_t)a.table.max_pages << shift;
            if (lead && c[u].bad) paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            if (lead && grows && !fits[u]) paged_flag(a.status, GRET_PAGED_TABLE_FULL);
            id[u] = -1;
            if (fits[u] && (c[u].n0 & ((1 << shift) - 1))) {
                id[u] = a.table.entries[(sb + u) * a.table.stride + (c[u].n0 >> shift)];
                if ((unsigned)id[u] >= (unsigned)a.pool.n_pages) {
                    if (lead) paged_flag(a.status, GRET_PAGED_BAD_PAGE);
                    id[u] = -1;
                    fits[u] = false;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) count[u] = id[u] >= 0 ? a.ref[id[u]] : 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = sb + u;
            if (s >= s1) break;
            if (count[u] <= 0) {                 // free, they say: this call may hand it out
                if (lead) paged_flag(a.status, GRET_PAGED_BAD_COUNT);
                fits[u] = false;
            }
            const int c0 = pages_of(c[u].n0, shift), c1 = pages_of(c[u].n1, shift);
            const bool copies = count[u] > 1;
            const int need = fits[u] ? c1 - c0 + copies : 0;
            upto[s] = need;
            first[s] = fits[u] ? c0 - copies : 0;
            if (lead) {
                a.workspace[s] = copies ? id[u] : -1;
                a.pos[s] = fits[u] ? (int)c[u].n0 : -1;
            }
            mine += need;
        }
    }
    return mine;
}

// The first of S rows with upto > rank (there is one), by a whole warp.
__device__ __forceinline__ int row_of_rank(const int* upto, int S, int rank) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = S;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool past = lane * step < n && (lane == 0 || upto[lo + lane * step - 1] <= rank);
        const int last = __popc(__ballot_sync(0xffffffffu, past)) - 1;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// Leaves pos, the new pages' ref and table entries, and in workspace[s] the page that row s is to
// copy its last, partly filled one from (-1: none).
template <int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(PNT, 1)
    resize_plan_kernel(const PagedResizeArgs a) {
    extern __shared__ int rows_smem[];
    __shared__ int64_t sums[PNW][2];
    __shared__ int chunk_before[MAXCH];
    int* upto = rows_smem;                        // [S] pages asked for by rows 0 .. s
    int* first = rows_smem + a.table.S;           // [S] table entry the first of them goes to
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    wait_for_previous();
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, S = a.table.S;
    const bool lead = cluster.block_rank() == 0;
    const int shift = a.pool.page_shift;

    // every block works out all rows' needs; the first one writes the plan
    const int per = (S + PNT - 1) / PNT;
    const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
    const int64_t mine = per == 1 ? needs_of<1>(a, s0, s1, lead, upto, first)
                                  : needs_of<4>(a, s0, s1, lead, upto, first);
    const Chunks ch(a.ref, a.pool.n_pages);
    count_free<CL>(ch, chunk_before);
    int64_t run = mine;
    const int total = rank_free(ch, chunk_before, sums, run);
    for (int s = s0; s < s1; ++s) {
        run += upto[s];
        upto[s] = (int)(run < INT_MAX ? run : INT_MAX);
    }
    __syncthreads();
    // rows up to `last` that ask for pages get them: upto rises, so the others follow
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] <= total) lo = mid + 1;
        else hi = mid;
    }
    const int granted = lo ? upto[lo - 1] : 0;
    if (lead)
        for (int s = max(lo, s0); s < s1; ++s) {   // the thread that wrote the row's plan
            const Change c = change_of(a, s);
            if (a.pos[s] >= 0 &&
                (a.workspace[s] >= 0 || pages_of(c.n1, shift) > pages_of(c.n0, shift))) {
                a.pos[s] = a.workspace[s] = -1;
                paged_flag(a.status, GRET_PAGED_NO_PAGES);
            }
        }
    // hand out the free pages of rank < granted
    const int warp = cluster.block_rank() * PNW + (tid >> 5);
    for (int c = warp; c < ch.n && chunk_before[c] < granted; c += CL * PNW) {
        int before = chunk_before[c];
        for (int q0 = c * ch.step; q0 < (c + 1) * ch.step && before < granted; q0 += 32) {
            const int4 x4 = ch.quad(q0 + lane);
            const int rank0 = before;
            const int4 rank4 = ranks_of(x4, before);
            if (before == rank0) continue;
            // the rows of these up to 128 pages, then each page's among them, four searches side by
            // side
            const int row0 = row_of_rank(upto, S, rank0);
            const int row1 = row_of_rank(upto, S, min(before, granted) - 1);
            const int x[4] = {x4.x, x4.y, x4.z, x4.w};
            const int rank[4] = {rank4.x, rank4.y, rank4.z, rank4.w};
            int l[4] = {row0, row0, row0, row0}, r[4] = {row1, row1, row1, row1};
            for (int n = row1 - row0; n > 0; n >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int mid = (l[u] + r[u]) >> 1;
                    if (upto[mid] > rank[u]) r[u] = mid;
                    else l[u] = min(mid + 1, row1);
                }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (x[u] != 0 || rank[u] >= granted) continue;
                const int at = ch.entry(q0 + lane) + u, row = r[u];
                a.table.entries[row * a.table.stride + first[row] + rank[u] -
                                (row ? upto[row - 1] : 0)] = at;
                a.ref[at] = 1;
            }
        }
    }
}

__device__ __forceinline__ void drop_page(const PagedResizeArgs& a, int id) {
    if (atomicSub(&a.ref[id], 1) <= 0) {
        atomicAdd(&a.ref[id], 1);
        paged_flag(a.status, GRET_PAGED_BAD_COUNT);
    }
}

// The entries [j0, j1) of a row, by the whole block: four a thread on their way at a time.
__device__ __forceinline__ void drop_entries(const PagedResizeArgs& a, int32_t* row, int j0,
                                             int j1) {
    constexpr int U = 4;
    for (int j = j0 + threadIdx.x; j < j1; j += NT * U) {
        int id[U], had[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = j + u * NT < j1 ? row[j + u * NT] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            had[u] = 1;
            if ((unsigned)id[u] < (unsigned)a.pool.n_pages) had[u] = atomicSub(&a.ref[id[u]], 1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u * NT >= j1) continue;
            row[j + u * NT] = -1;
            if ((unsigned)id[u] >= (unsigned)a.pool.n_pages) {
                paged_flag(a.status, GRET_PAGED_BAD_PAGE);
            } else if (had[u] <= 0) {
                atomicAdd(&a.ref[id[u]], 1);
                paged_flag(a.status, GRET_PAGED_BAD_COUNT);
            }
        }
    }
}

__global__ void __launch_bounds__(NT, APPLY_SM) resize_apply_kernel(const PagedResizeArgs a,
                                                                    const Pieces pc) {
    constexpr int GRID = APPLY_SM * 148;
    __shared__ int from[NT], to[NT], slots[NT], in_warp[NT / 32];
    const int tid = threadIdx.x, S = a.table.S, shift = a.pool.page_shift;
    wait_for_previous();
    // a block a row: pages that it drops, its new length
    for (int s = blockIdx.x; s < S; s += GRID) {
        const Change c = change_of(a, s);
        const bool grown = a.pos[s] >= 0, shrunk = !c.bad && c.n1 < c.n0;
        if (shrunk) {
            drop_entries(a, a.table.entries + s * a.table.stride, pages_of(c.n1, shift),
                         pages_of(c.n0, shift));
        } else if (grown && tid == 0 && a.workspace[s] >= 0) {
            drop_page(a, a.workspace[s]);
        }
        __syncthreads();   // every thread has read the length
        if (tid == 0 && (grown || shrunk)) a.seq_lens[s] = (int)c.n1;
    }
    // the copies, NT rows at a time, in steps dealt over all blocks.  pos is the old length
    const int steps = (pc.total + NT - 1) / NT;
    int k = blockIdx.x / steps, c = blockIdx.x % steps;   // next: step c of the batch's row k
    const int dk = GRID / steps, dc = GRID % steps;
    for (int s0 = 0; s0 < S; s0 += NT) {
        // the batch's rows that copy, in order: all blocks have to count them alike
        const int s = s0 + tid, src = s < S ? a.workspace[s] : -1;
        const unsigned mask = __ballot_sync(0xffffffffu, src >= 0);
        __syncthreads();                          // the batch before is done with
        if ((tid & 31) == 0) in_warp[tid >> 5] = __popc(mask);
        __syncthreads();
        int x = __popc(mask & ((1u << (tid & 31)) - 1)), copies = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < (tid >> 5)) x += in_warp[w];
            copies += in_warp[w];
        }
        if (src >= 0) {
            const int n0 = a.pos[s];
            from[x] = src;
            to[x] = a.table.entries[s * a.table.stride + (n0 >> shift)];
            slots[x] = n0 & ((1 << shift) - 1);
        }
        __syncthreads();
        while (k < copies) {
            if (pc.tokens_inside || c * NT < slots[k] * (int)pc.outer.d)
                copy_pieces(a.pool, pc, from[k], to[k], c * NT, slots[k]);
            k += dk;
            c += dc;
            if (c >= steps) {
                c -= steps;
                ++k;
            }
        }
        k -= copies;
    }
}

// ---------------------------------------------------------------------------------------------
// fork.  Bound by latency: 64 rows of 50 entries take 2.8 us, 512 of 7000 11.8, of which the copy of
// the 14 MB of entries would take 2.2.  The rest is the chain of every block before its first entry
// (the pairs, the rows that they name, their lengths; and once more over all pairs for those that
// share a source), then that of the second kernel.  Counts of pages that many rows share would be
// bound by atomics on one address if each pair added its 1: there, of the m pairs of a source each
// adds m to an m-th of its pages.  That takes the pairs' knowing of one another, so that the lengths,
// by which a pair that has no effect is known, can only be set by a second kernel; small calls go
// without.

// The first pair that names each row as its destination (INT_MAX: none).
__device__ __forceinline__ void first_pairs(const PagedForkArgs& a, int* first) {
    for (int s = threadIdx.x; s < a.table.S; s += NT) first[s] = INT_MAX;
    __syncthreads();
    for (int j = threadIdx.x; j < a.n; j += NT) {
        const int d = a.dst[j];
        if ((unsigned)d < (unsigned)a.table.S) atomicMin(&first[d], j);
    }
    __syncthreads();
}

// Whether pair j takes effect.  seq_lens as before the call.
__device__ __forceinline__ bool takes_effect(const PagedForkArgs& a, const int* first, int j) {
    const int s = a.src[j], d = a.dst[j], S = a.table.S;
    if ((unsigned)s >= (unsigned)S || (unsigned)d >= (unsigned)S) return false;
    const int n = a.seq_lens[s];
    return first[d] == j && first[s] == INT_MAX && a.seq_lens[d] == 0 && n >= 0 &&
           n <= (int64_t)a.table.max_pages << a.page_shift;
}

template <bool SHARE>
__global__ void __launch_bounds__(NT) fork_kernel(const PagedForkArgs a) {
    extern __shared__ int first[];
    __shared__ int before[NT / 32], siblings[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_previous();
    if (SHARE) let_next_start();
    first_pairs(a, first);
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        if (!takes_effect(a, first, i)) {
            if (blockIdx.y == 0 && tid == 0) paged_flag(a.status, GRET_PAGED_BAD_ROW);
            continue;
        }
        const int s = a.src[i], d = a.dst[i], n = a.seq_lens[s];
        const int held = pages_of(n, a.page_shift);
        int lo = 0, hi = held, add = 1;           // the entries whose pages it counts
        if (SHARE) {
            int k = 0, m = 0;                     // pairs of this source before i, and in all
            for (int j = tid; j < a.n; j += NT)
                if (a.src[j] == s && takes_effect(a, first, j)) {
                    ++m;
                    k += j < i;
                }
            k = __reduce_add_sync(0xffffffffu, k);
            m = __reduce_add_sync(0xffffffffu, m);
            __syncthreads();
            if (lane == 0) {
                before[warp] = k;
                siblings[warp] = m;
            }
            __syncthreads();
            k = m = 0;
            for (int w = 0; w < NT / 32; ++w) {
                k += before[w];
                m += siblings[w];
            }
            lo = (int)((int64_t)held * k / m);
            hi = (int)((int64_t)held * (k + 1) / m);
            add = m;
        }
        const int32_t* from = a.table.entries + s * a.table.stride;
        int32_t* to = a.table.entries + d * a.table.stride;
        constexpr int U = 4;
        for (int j0 = blockIdx.y * NT * U; j0 < held; j0 += gridDim.y * NT * U) {
            int id[U], had[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * NT + tid;
                if (j < held) id[u] = from[j];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * NT + tid;
                had[u] = 1;
                if (j >= held) continue;
                to[j] = id[u];
                if (j < lo || j >= hi) continue;
                // the old count is asked for where it can be reported: additions that return it take
                // a third longer (512 rows of 512 entries, 2 of a source, 3.9 -> 5.1 us)
                if ((unsigned)id[u] >= (unsigned)a.n_pages) paged_flag(a.status, GRET_PAGED_BAD_PAGE);
                else if (!a.status) atomicAdd(&a.ref[id[u]], add);
                else had[u] = atomicAdd(&a.ref[id[u]], add);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (had[u] <= 0) paged_flag(a.status, GRET_PAGED_BAD_COUNT);
        }
        if (!SHARE) {
            __syncthreads();                      // every thread has read the lengths
            if (tid == 0) a.seq_lens[d] = n;
        }
    }
}

// The destinations' lengths, once nobody asks any more whether they are empty.
__global__ void __launch_bounds__(NT) fork_lengths_kernel(const PagedForkArgs a) {
    extern __shared__ int first[];
    wait_for_previous();
    first_pairs(a, first);
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i < a.n && takes_effect(a, first, i)) a.seq_lens[a.dst[i]] = a.seq_lens[a.src[i]];
}

// ---------------------------------------------------------------------------------------------
// compact: with L pages in use, the k-th page in use past L moves to the k-th hole below L.  Bound
// by HBM but for small pools: 16400 pages of 64 KB moved in 338 us (6.3 TB/s), 240 in 11.

// The plan in the workspace: {L, pages to move}, then by page: the k-th hole, the page in use of
// rank r (of those past L), the rank of a page in use (-1: free).
struct CompactPlan {
    int32_t *counts, *holes, *used, *rank;
};

__host__ __device__ __forceinline__ CompactPlan compact_plan(const PagedCompactArgs& a) {
    const int64_t P = a.pool.n_pages;
    return {a.workspace, a.workspace + 4, a.workspace + 4 + P, a.workspace + 4 + 2 * P};
}

template <int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(PNT, 1)
    compact_plan_kernel(const PagedCompactArgs a) {
    __shared__ int64_t sums[PNW][2];
    __shared__ int chunk_before[MAXCH];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    wait_for_previous();
    let_next_start();
    const int lane = threadIdx.x & 31, P = a.pool.n_pages;
    const CompactPlan plan = compact_plan(a);
    const Chunks ch(a.ref, P);
    count_free<CL>(ch, chunk_before);
    int64_t none = 0;
    const int L = P - rank_free(ch, chunk_before, sums, none);
    __syncthreads();
    if (cluster.block_rank() == 0 && threadIdx.x == 0) {
        *a.n_live = L;
        plan.counts[0] = L;
        if (L == P) plan.counts[1] = 0;            // no page has the index L
    }
    for (int c = cluster.block_rank() * PNW + (threadIdx.x >> 5); c < ch.n; c += CL * PNW) {
        int before = chunk_before[c];
        for (int q0 = c * ch.step; q0 < (c + 1) * ch.step; q0 += 32) {
            const int4 x4 = ch.quad(q0 + lane), h4 = ranks_of(x4, before);
            const int x[4] = {x4.x, x4.y, x4.z, x4.w}, h[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = ch.entry(q0 + lane) + u;
                if (at < 0 || at >= P) continue;
                if (at == L) plan.counts[1] = h[u];    // holes below L = pages in use past it
                plan.rank[at] = x[u] == 0 ? -1 : at - h[u];
                if (at < L && x[u] == 0) plan.holes[h[u]] = at;
                if (at >= L && x[u] != 0) plan.used[at - h[u]] = at;
            }
        }
    }
}

__global__ void __launch_bounds__(NT) compact_move_kernel(const PagedCompactArgs a,
                                                          const Pieces pc) {
    const CompactPlan plan = compact_plan(a);
    wait_for_previous();
    const int L = plan.counts[0], moves = plan.counts[1];
    // step c of move k, dealt over the blocks.  The counts move apart from the pages: a thread that
    // waits for a count inside this loop holds its block's next step up (332 -> 388 us for 16448
    // moves of 64 KB)
    const int steps = (pc.total + NT - 1) / NT;
    int k = blockIdx.x / steps, c = blockIdx.x % steps;
    const int dk = GRID / steps, dc = GRID % steps;
    while (k < moves) {
        const int from = plan.used[L - moves + k], to = plan.holes[k];
        copy_pieces(a.pool, pc, from, to, c * NT, 1 << a.pool.page_shift);
        k += dk;
        c += dc;
        if (c >= steps) {
            c -= steps;
            ++k;
        }
    }
    for (k = blockIdx.x * NT + threadIdx.x; k < moves; k += GRID * NT) {
        const int from = plan.used[L - moves + k];
        a.ref[plan.holes[k]] = a.ref[from];
        a.ref[from] = 0;
    }
    const int64_t cap = (int64_t)a.table.max_pages << a.pool.page_shift;
    for (int s = blockIdx.x; s < a.table.S; s += GRID) {
        const int64_t n = a.seq_lens[s];
        if (n < 0 || n > cap) {
            if (threadIdx.x == 0) paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            continue;
        }
        int32_t* row = a.table.entries + s * a.table.stride;
#pragma unroll 4
        for (int j = threadIdx.x; j < pages_of(n, a.pool.page_shift); j += NT) {
            const int id = row[j];
            if ((unsigned)id >= (unsigned)a.pool.n_pages) {
                paged_flag(a.status, GRET_PAGED_BAD_PAGE);
                continue;
            }
            const int r = plan.rank[id];       // as of before the moves, for pages below L too
            if (r < 0) paged_flag(a.status, GRET_PAGED_BAD_COUNT);
            else if (id >= L) row[j] = plan.holes[r - (L - moves)];
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
    // one token a warp up to a full GPU of warps (148 x 64), then more of them
    const int64_t even = a.T / (148 * 64);
    const int tok = (int)(even < 1 ? 1 : even > AP_MAXTOK ? AP_MAXTOK : even);
    const int64_t per = (int64_t)(NT / 32) * tok;
    const uint32_t row = a.pool.row_bytes / 16;
    return launch_early(append_kernel, dim3((unsigned)((a.T + per - 1) / per)), NT, 0, stream, a,
                        FastDiv(a.pool.H * row), FastDiv(row), tok);
}

cudaError_t launch_paged_resize(const PagedResizeArgs& a, cudaStream_t stream) {
    const size_t smem = (size_t)a.table.S * 2 * sizeof(int);
    constexpr int most_smem = PAGED_MAX_SEQS * 2 * (int)sizeof(int);
    cudaError_t e;
    if (a.pool.n_pages >= MANY_PAGES && many_blocks<resize_plan_kernel<CL_MANY>>(most_smem)) {
        e = launch_early(resize_plan_kernel<CL_MANY>, dim3(CL_MANY), PNT, smem, stream, a);
    } else {
        e = allow_smem<resize_plan_kernel<CL_FEW>>(smem, most_smem);
        if (e == cudaSuccess)
            e = launch_early(resize_plan_kernel<CL_FEW>, dim3(CL_FEW), PNT, smem, stream, a);
    }
    if (e != cudaSuccess) return e;
    return launch_early(resize_apply_kernel, dim3(APPLY_SM * 148), NT, 0, stream, a,
                        Pieces(a.pool));
}

cudaError_t launch_paged_fork(const PagedForkArgs& a, cudaStream_t stream) {
    constexpr int most_smem = PAGED_MAX_SEQS * (int)sizeof(int);
    const size_t smem = (size_t)a.table.S * sizeof(int);
    const int x = a.n < 2 * GRID ? a.n : 2 * GRID;
    cudaError_t e;
    // Without sharing out the counts: one launch, a block a pair.  Measured against two launches, in
    // us, for 2, 8 and 125 rows a source: 64 rows of 76 entries 2.6, 2.8, 2.9 and 5.1, 5.4, 5.5; 512 of
    // 512 3.9, 5.3, 13.5 and 6.6, 7.2, 7.4; 2000 of 1000 17, 17, 33 and 19, 16, 19; 1024 of 2040 15, 16,
    // 30 and 14, 11, 10; 512 of 8180 30, 30, 48 and 21, 15, 12; and one row of 32768, which only the
    // other cuts up, 26 and 6.  How many rows share a source the host does not know: the rule is for
    // few.
    if (a.table.max_pages <= 8192 && (int64_t)a.n * a.table.max_pages <= FORK_ALONE) {
        e = allow_smem<fork_kernel<false>>(smem, most_smem);
        if (e != cudaSuccess) return e;
        return launch_early(fork_kernel<false>, dim3(x), NT, smem, stream, a);
    }
    e = allow_smem<fork_kernel<true>>(smem, most_smem);
    if (e == cudaSuccess) e = allow_smem<fork_lengths_kernel>(smem, most_smem);
    if (e != cudaSuccess) return e;
    // a block a pair; with few pairs a row is cut up, in pieces of 1024 entries or more
    int y = 2 * GRID / x, most = (a.table.max_pages + 1023) / 1024;
    if (y > most) y = most;
    e = launch_early(fork_kernel<true>, dim3(x, y), NT, smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_early(fork_lengths_kernel, dim3((a.n + NT - 1) / NT), NT, smem, stream, a);
}

cudaError_t launch_paged_compact(const PagedCompactArgs& a, cudaStream_t stream) {
    const cudaError_t e = launch_early(compact_plan_kernel<CL_FEW>, dim3(CL_FEW), PNT, 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_early(compact_move_kernel, dim3(GRID), NT, 0, stream, a, Pieces(a.pool));
}

}  // namespace gret
