// paged_cache.cu -- the upkeep of a paged key-value cache: writing new tokens, growing and
// shrinking sequences with copy on write, sharing pages with a new sequence, compaction.
//
// Which pages are free is ref[p] == 0, nothing else: no free list to keep in step.  A call that
// takes pages takes the lowest free ones, row after row, so the outcome depends on the inputs
// alone.  Finding them is a ranking of the free pages (how many free pages lie below p), which a
// cluster of CL blocks does in one launch: every warp counts a contiguous slice of ref by ballots,
// the blocks exchange their counts through distributed shared memory, and a second walk over a
// slice, only by warps that need it, hands out the ranks.
#include <limits.h>

#include <cooperative_groups.h>

#include "common.cuh"
#include "paged.cuh"

namespace gret {

namespace cg = cooperative_groups;

namespace {

constexpr int CL = 8;                  // blocks of a planning cluster (the portable maximum)
constexpr int PNT = 1024;
constexpr int PNW = PNT / 32;

// Exclusive sum of x over the block's threads, and the total.  `sums` has PNW entries.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before + incl - x;
}

// The slice of ref that a warp of the cluster ranks.
struct Slice {
    int lo, hi;
};

__device__ __forceinline__ Slice warp_slice(int n_pages, int rank) {
    const int64_t warps = CL * PNW, w = rank * PNW + (threadIdx.x >> 5);
    const int64_t step = ((n_pages + warps - 1) / warps + 31) / 32 * 32;
    const int64_t lo = w * step, hi = lo + step;
    return {(int)(lo < n_pages ? lo : n_pages), (int)(hi < n_pages ? hi : n_pages)};
}

// Free pages of the slice, counted by the whole warp.
__device__ __forceinline__ int count_free(const int32_t* ref, Slice s) {
    int n = 0;
    for (int i = s.lo; i < s.hi; i += 32) {
        const int at = i + (threadIdx.x & 31);
        n += __popc(__ballot_sync(0xffffffffu, at < s.hi && ref[at] == 0));
    }
    return n;
}

// Free pages before this warp's slice, and in all of the pool.  Ends with a cluster barrier: all
// blocks' counts are taken.
__device__ __forceinline__ void rank_free(int mine, int* warp_free, int* block_free, int& before,
                                          int& total) {
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) warp_free[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < PNW; ++w) n += warp_free[w];
        *block_free = n;
    }
    cluster.sync();
    before = total = 0;
    for (unsigned r = 0; r < CL; ++r) {
        const int n = *cluster.map_shared_rank(block_free, r);
        if (r < cluster.block_rank()) before += n;
        total += n;
    }
    for (int w = 0; w < warp; ++w) before += warp_free[w];
}

// ---------------------------------------------------------------------------------------------
// append: a copy of every token's row of heads to its slot.

constexpr int AP_NT = 256;
constexpr int AP_TOK = 8;              // tokens a warp takes one after another

__global__ void __launch_bounds__(AP_NT) append_kernel(const PagedAppendArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t i0 = ((int64_t)blockIdx.x * (AP_NT / 32) + (threadIdx.x >> 5)) * AP_TOK;
    const int64_t cap = (int64_t)a.table.max_pages << a.pool.page_shift;
    const int cpr = a.pool.row_bytes / 16;       // 16-byte pieces of a row
    int b = 0;
    if (a.cu_seqlens) {                           // the last row that begins at or before i0
        int hi = a.table.S - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (a.cu_seqlens[mid] <= i0) b = mid;
            else hi = mid - 1;
        }
    }
    for (int64_t i = i0; i < i0 + AP_TOK && i < a.T; ++i) {
        int64_t at;
        if (a.cu_seqlens) {
            while (b < a.table.S && a.cu_seqlens[b + 1] <= i) ++b;
            if (b == a.table.S) return;           // behind the last sequence
            if (i < a.cu_seqlens[b]) continue;    // before the first one
            at = i - a.cu_seqlens[b];
        } else {
            b = (int)i;
            at = 0;
        }
        const int pos = a.pos[b];
        if (pos < 0) continue;
        at += pos;
        if (at >= cap) {
            if (lane == 0) paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            continue;
        }
        const int id = a.table.entries[b * a.table.stride + (at >> a.pool.page_shift)];
        if ((unsigned)id >= (unsigned)a.pool.n_pages) {
            if (lane == 0) paged_flag(a.status, GRET_PAGED_BAD_PAGE);
            continue;
        }
        const int64_t slot = id * a.pool.sp + (at & ((1 << a.pool.page_shift) - 1)) * a.pool.st;
        for (int c = lane; c < a.pool.H * cpr; c += 32) {
            const int h = c / cpr, x = (c % cpr) * 16;
            const uint4 kx = *reinterpret_cast<const uint4*>(a.k + i * a.kt + h * a.kh + x);
            const uint4 vx = *reinterpret_cast<const uint4*>(a.v + i * a.vt + h * a.vh + x);
            *reinterpret_cast<uint4*>(a.pool.k + slot + h * a.pool.sh + x) = kx;
            *reinterpret_cast<uint4*>(a.pool.v + slot + h * a.pool.sh + x) = vx;
        }
    }
}

// Slots [0, slots) of page `from` to page `to`, by the whole block.
__device__ __forceinline__ void copy_slots(const PagedPool& p, int64_t from, int64_t to, int slots) {
    const int cpr = p.row_bytes / 16, per = p.H * cpr;
    for (int c = threadIdx.x; c < slots * per; c += blockDim.x) {
        const int t = c / per, h = c % per / cpr;
        const int64_t off = t * p.st + h * p.sh + (c % cpr) * 16;
        const uint4 kx = *reinterpret_cast<const uint4*>(p.k + from * p.sp + off);
        const uint4 vx = *reinterpret_cast<const uint4*>(p.v + from * p.sp + off);
        *reinterpret_cast<uint4*>(p.k + to * p.sp + off) = kx;
        *reinterpret_cast<uint4*>(p.v + to * p.sp + off) = vx;
    }
}

// ---------------------------------------------------------------------------------------------
// resize: a plan by one cluster (who gets which page), then one block a row carries it out.

// What the plan says of a row that grows; else it holds the page to copy from.
enum : int { PLAN_NO_COPY = -1, PLAN_REFUSED = -2 };

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

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(PNT)
    resize_plan_kernel(const PagedResizeArgs a) {
    extern __shared__ int rows_smem[];
    __shared__ int64_t sums[PNW];
    __shared__ int warp_free[PNW], block_free;
    int* upto = rows_smem;                        // [S] pages asked for by rows 0 .. s
    int* first = rows_smem + a.table.S;           // [S] table entry the first of them goes to
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, S = a.table.S;
    const bool lead = cluster.block_rank() == 0;
    const int shift = a.pool.page_shift;

    // every block works out all rows' needs; the first one writes the plan
    const int per = (S + PNT - 1) / PNT;
    const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        const Change c = change_of(a, s);
        int need = 0, src = PLAN_NO_COPY;
        first[s] = 0;
        if (c.bad) {
            if (lead) paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            src = PLAN_REFUSED;
        } else if (c.n1 > c.n0) {
            if (c.n1 > (int64_t)a.table.max_pages << shift) {
                if (lead) paged_flag(a.status, GRET_PAGED_TABLE_FULL);
                src = PLAN_REFUSED;
            } else {
                const int c0 = pages_of(c.n0, shift), c1 = pages_of(c.n1, shift);
                if (c.n0 & ((1 << shift) - 1)) {
                    const int id = a.table.entries[s * a.table.stride + c0 - 1];
                    if ((unsigned)id >= (unsigned)a.pool.n_pages) {
                        if (lead) paged_flag(a.status, GRET_PAGED_BAD_PAGE);
                    } else if (a.ref[id] > 1) {
                        src = id;
                    }
                }
                need = c1 - c0 + (src >= 0);
                first[s] = c0 - (src >= 0);
            }
        }
        upto[s] = need;
        if (lead) a.workspace[s] = src;
        mine += need;
    }
    int64_t asked;
    int64_t run = block_scan(mine, sums, asked);
    for (int s = s0; s < s1; ++s) {
        run += upto[s];
        upto[s] = (int)(run < INT_MAX ? run : INT_MAX);
    }
    const Slice slice = warp_slice(a.pool.n_pages, cluster.block_rank());
    int before, total;
    rank_free(count_free(a.ref, slice), warp_free, &block_free, before, total);
    // rows up to `last` that ask for pages get them: upto rises, so the others follow
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] <= total) lo = mid + 1;
        else hi = mid;
    }
    const int granted = lo ? upto[lo - 1] : 0;
    if (lead)
        for (int s = lo + tid; s < S; s += PNT) {
            const Change c = change_of(a, s);
            const int src = a.workspace[s];
            if (c.n1 > c.n0 && src != PLAN_REFUSED &&
                (src >= 0 || pages_of(c.n1, shift) > pages_of(c.n0, shift))) {
                a.workspace[s] = PLAN_REFUSED;
                paged_flag(a.status, GRET_PAGED_NO_PAGES);
            }
        }
    // hand out the free pages of rank < granted
    for (int i = slice.lo; i < slice.hi && before < granted; i += 32) {
        const int at = i + lane;
        const bool free = at < slice.hi && a.ref[at] == 0;
        const unsigned mask = __ballot_sync(0xffffffffu, free);
        const int rank = before + __popc(mask & ((1u << lane) - 1));
        if (free && rank < granted) {
            int l = 0, r = S - 1;                 // the first row with upto > rank
            while (l < r) {
                const int mid = (l + r) >> 1;
                if (upto[mid] > rank) r = mid;
                else l = mid + 1;
            }
            a.table.entries[l * a.table.stride + first[l] + rank - (l ? upto[l - 1] : 0)] = at;
            a.ref[at] = 1;
        }
        before += __popc(mask);
    }
    cluster.sync();   // no block leaves while another reads its count
}

__global__ void __launch_bounds__(256) resize_apply_kernel(const PagedResizeArgs a) {
    const int s = blockIdx.x, shift = a.pool.page_shift;
    const Change c = change_of(a, s);
    const int plan = a.workspace[s];
    int32_t* row = a.table.entries + s * a.table.stride;
    const int c0 = pages_of(c.n0, shift);
    bool done = false;
    if (!c.bad && c.n1 > c.n0 && plan != PLAN_REFUSED) {
        done = true;
        if (plan >= 0) {
            copy_slots(a.pool, plan, row[c0 - 1], (int)(c.n0 & ((1 << shift) - 1)));
            if (threadIdx.x == 0 && atomicSub(&a.ref[plan], 1) <= 0) {
                atomicAdd(&a.ref[plan], 1);
                paged_flag(a.status, GRET_PAGED_BAD_COUNT);
            }
        }
    } else if (!c.bad && c.n1 < c.n0) {
        for (int j = pages_of(c.n1, shift) + threadIdx.x; j < c0; j += blockDim.x) {
            const int id = row[j];
            row[j] = -1;
            if ((unsigned)id >= (unsigned)a.pool.n_pages) {
                paged_flag(a.status, GRET_PAGED_BAD_PAGE);
            } else if (atomicSub(&a.ref[id], 1) <= 0) {
                atomicAdd(&a.ref[id], 1);
                paged_flag(a.status, GRET_PAGED_BAD_COUNT);
            }
        }
    }
    __syncthreads();   // every thread has read the length
    if (threadIdx.x == 0) {
        a.pos[s] = done ? (int)c.n0 : -1;
        if (done || (!c.bad && c.n1 < c.n0)) a.seq_lens[s] = (int)c.n1;
    }
}

// ---------------------------------------------------------------------------------------------
// fork: one block a pair.

__global__ void __launch_bounds__(256) fork_kernel(const PagedForkArgs a) {
    const int i = blockIdx.x, S = a.table.S;
    const int s = a.src[i], d = a.dst[i];
    bool bad = (unsigned)s >= (unsigned)S || (unsigned)d >= (unsigned)S || s == d;
    // refused: a destination that an earlier pair names, a source that is a destination
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) {
        const int x = a.dst[j];
        bad |= (j < i && x == d) || x == s;
    }
    int64_t n = 0;
    if (!__syncthreads_or(bad)) {
        n = a.seq_lens[s];
        bad = a.seq_lens[d] != 0 || n < 0 || n > (int64_t)a.table.max_pages << a.page_shift;
    } else {
        bad = true;
    }
    __syncthreads();   // every thread has read the lengths
    if (bad) {
        if (threadIdx.x == 0) paged_flag(a.status, GRET_PAGED_BAD_ROW);
        return;
    }
    const int held = pages_of(n, a.page_shift);
    for (int j = threadIdx.x; j < held; j += blockDim.x) {
        const int id = a.table.entries[s * a.table.stride + j];
        a.table.entries[d * a.table.stride + j] = id;
        if ((unsigned)id < (unsigned)a.n_pages) atomicAdd(&a.ref[id], 1);
        else paged_flag(a.status, GRET_PAGED_BAD_PAGE);
    }
    if (threadIdx.x == 0) a.seq_lens[d] = (int)n;
}

// ---------------------------------------------------------------------------------------------
// compact: with L pages in use, the k-th page in use past L moves to the k-th hole below L.

// The plan in the workspace: {L, pages to move}, then by page: the k-th hole, the page in use of
// rank r, the rank of a page in use past L (-1: free).
struct CompactPlan {
    int32_t *counts, *holes, *used, *rank;
};

__host__ __device__ __forceinline__ CompactPlan compact_plan(const PagedCompactArgs& a) {
    const int64_t P = a.pool.n_pages;
    return {a.workspace, a.workspace + 4, a.workspace + 4 + P, a.workspace + 4 + 2 * P};
}

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(PNT)
    compact_plan_kernel(const PagedCompactArgs a) {
    __shared__ int warp_free[PNW], block_free;
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, P = a.pool.n_pages;
    const CompactPlan plan = compact_plan(a);
    const Slice slice = warp_slice(P, cluster.block_rank());
    int holes, total;                              // free pages before the one at hand
    rank_free(count_free(a.ref, slice), warp_free, &block_free, holes, total);
    const int L = P - total;
    if (cluster.block_rank() == 0 && threadIdx.x == 0) {
        *a.n_live = L;
        plan.counts[0] = L;
        if (L == P) plan.counts[1] = 0;            // no page has the index L
    }
    for (int i = slice.lo; i < slice.hi; i += 32) {
        const int at = i + lane;
        const bool free = at < slice.hi && a.ref[at] == 0;
        const unsigned mask = __ballot_sync(0xffffffffu, free);
        const int h = holes + __popc(mask & ((1u << lane) - 1));
        if (at < slice.hi) {
            if (at == L) plan.counts[1] = h;       // holes below L = pages in use past it
            if (at < L) {
                if (free) plan.holes[h] = at;
            } else {
                plan.rank[at] = free ? -1 : at - h;
                if (!free) plan.used[at - h] = at;
            }
        }
        holes += __popc(mask);
    }
    cluster.sync();   // no block leaves while another reads its count
}

__global__ void __launch_bounds__(256) compact_move_kernel(const PagedCompactArgs a) {
    const CompactPlan plan = compact_plan(a);
    const int L = plan.counts[0], moves = plan.counts[1];
    for (int k = blockIdx.x; k < moves; k += gridDim.x) {
        const int from = plan.used[L - moves + k], to = plan.holes[k];
        copy_slots(a.pool, from, to, 1 << a.pool.page_shift);
        if (threadIdx.x == 0) {
            a.ref[to] = a.ref[from];
            a.ref[from] = 0;
        }
    }
    const int64_t cap = (int64_t)a.table.max_pages << a.pool.page_shift;
    for (int s = blockIdx.x; s < a.table.S; s += gridDim.x) {
        const int64_t n = a.seq_lens[s];
        if (n < 0 || n > cap) {
            if (threadIdx.x == 0) paged_flag(a.status, GRET_PAGED_BAD_LENGTH);
            continue;
        }
        int32_t* row = a.table.entries + s * a.table.stride;
        for (int j = threadIdx.x; j < pages_of(n, a.pool.page_shift); j += blockDim.x) {
            const int id = row[j];
            if ((unsigned)id >= (unsigned)a.pool.n_pages) {
                paged_flag(a.status, GRET_PAGED_BAD_PAGE);
            } else if (id >= L) {
                const int r = plan.rank[id];
                if (r < 0) paged_flag(a.status, GRET_PAGED_BAD_COUNT);
                else row[j] = plan.holes[r - (L - moves)];
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
    const int64_t per = (int64_t)(AP_NT / 32) * AP_TOK;
    append_kernel<<<(unsigned)((a.T + per - 1) / per), AP_NT, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_resize(const PagedResizeArgs& a, cudaStream_t stream) {
    const size_t smem = (size_t)a.table.S * 2 * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(resize_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PAGED_MAX_SEQS * 2 * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    resize_plan_kernel<<<CL, PNT, smem, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    resize_apply_kernel<<<(unsigned)a.table.S, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_fork(const PagedForkArgs& a, cudaStream_t stream) {
    fork_kernel<<<(unsigned)a.n, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_compact(const PagedCompactArgs& a, cudaStream_t stream) {
    compact_plan_kernel<<<CL, PNT, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    compact_move_kernel<<<148 * 4, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gret
