// paged_attention.cu -- attention of one new token over a paged key-value cache.
//
// Per sequence b and query head i, with n = seq_lens[b] keys (the last `window` of them where a
// window is given) and kv head h = i / (Hq / Hkv):
//     s_j = scale q . k_j,   m = max_j s_j,   l = sum_j e^(s_j - m),
//     o = sum_j e^(s_j - m) v_j / l,   lse = m + ln l.
// Parts of the keys give (m_i, l_i, a_i = sum e^(s_j - m_i) v_j), which join exactly:
//     m = max m_i,  l = sum e^(m_i - m) l_i,  o = sum e^(m_i - m) a_i / l.
//
// Bound: HBM, 2 n d values a (sequence, kv head) read once, 2 G flops a value.  That little
// arithmetic leaves the tensor cores idle for most of the time in any form (18 % busy at G = 3),
// so the form is chosen for the loads: every warp runs its own ring of cp.async tiles (KT keys and
// values of one head, 8 KB), all but one of them always in flight behind the one being worked on
// and across the borders of sequences, with no barrier between warps but where a (sequence, head)
// ends; page-table entries are read as many tiles ahead of that.  A ring has three tiles, of two
// blocks an SM (F32Math::MORE: two tiles, three blocks).  16-byte pieces gathered by lanes take
// any page size and any stride, where a bulk copy would want one tensor map a layout and at least
// a page of tokens. Measured, 8 kv heads of 128 in bf16, G = 3: 64 sequences of 200 to 32768
// tokens 266 to 272 us (6.5 TB/s, what a plain copy reaches), 2 of 524288 646 us; one of 4096 8.9
// us, of which 6.8 go by with no more than 100 tokens: two launches, and the chain length -> page
// -> keys -> parts -> join.
//
// bf16: keys are the M side of the product and the query heads of the group the N side (8 to 24,
// padded to a multiple of 8), S^T = K Q^T, so 3 heads cost 8 columns and not 16 rows; and O^T =
// V^T P^T with p cut into three bf16 parts of 8 bits, which together are p: the weights enter the
// product as they are summed up, in fp32.  Each 16 keys' products are summed up from 0 and added
// to the rest by the warp: a tensor core cuts its sums off, so that a long one in its accumulators
// falls short by 2^-23 or so of itself a step (65536 keys, 16384 a warp, 2048 steps: all outputs
// too small by 1.1e-4).  The third part takes 1 to 8 % of the time, these sums 0 to 15 (the more
// rows the more).  Keys and values are read from shared memory by ldmatrix, the sums stay in
// registers.  From 9 heads a group on the products and the softmax no longer hide behind the
// loads: 12 of 128 on each of two kv heads run at 0.71 of the copy bandwidth, 24 on one at 0.47,
// 32 (keys read twice) at 0.33. fp32: products in packed fp32 on the CUDA cores, a lane a key for
// the scores and a lane four dimensions for the values; 0.95 of the copy bandwidth at G = 3, 0.85
// at 8; at 16 (0.47) the queries' reads from shared memory bound it.
//
// The work is cut into units of UNIT keys of one (sequence, kv head, group of query rows), a pair;
// the units of the whole batch are dealt out evenly over the grid, in order, so that one long
// sequence spreads over every SM and a ragged batch stays balanced without the host knowing the
// lengths.  A block whose range ends inside a (sequence, head) writes its part to the workspace; a
// second kernel joins the parts in block order, so that results do not depend on timing.  Batches
// of many short pairs go to single warps instead (ByWarps).
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace gret {

namespace {

constexpr int NT = 128;
constexpr int NW = NT / 32;
constexpr int UNIT = 32;               // keys of one unit of work
// Pairs of up to so many tiles are worked on by single warps, where there are at least so many of
// them: half of the GPU's 1184 warps.  By warps and by blocks, in us: 640 pairs of 5 to 20 keys 8.7
// and 11.0, of 100 to 128 15.6 and 17.3; but 320 pairs of 100 to 128 keys 14.7 and 11.2.
constexpr int SHORT_TILES = 8;
constexpr int MIN_SHORT = 592;
constexpr int HALF = 4096;             // bytes of a tile's keys, and of its values
constexpr int STAGE = 2 * HALF;
constexpr int MAXROWS_BF16 = 24;       // query rows a block works on at a time: what registers hold
constexpr int MAXROWS_F32 = 16;
constexpr int MAX_GRID = 148 * 3;
// Blocks a pair of the join.  With 2, 4, 8 and 16 of them, calls in us: one sequence of 4096 keys
// (3 rows a pair) 10.4, 8.9 and no more change; 64 ragged ones of 24 heads on one kv head 84, 77, 75
// and 74.
constexpr int JOIN_Y = 8;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// What the join needs of block c: of the pair whose first part block c holds, and not the rest, the
// first query row, the rows, and the blocks that hold parts of it (block c's tail slot, then the
// head slots of the next).  No such pair: no rows.
struct Header {
    int32_t head;
    int16_t rows, parts;
};

// Parts in the workspace: slot 2c is block c's head (the rest of a pair begun by an earlier
// block), slot 2c + 1 its tail (a pair that a later block goes on with).
template <int MR, int R, int D>
struct Part {
    float m[MR], l[MR];            // m in units of log2
    float a[R][D];
};

struct Params {
    const void* q;
    const int32_t* lens;
    PagedTable table;
    PagedPool pool;
    float scale_log2;
    int window, Hq, G, QG;       // query heads a kv head; groups of rows of them
    void* o;
    float* lse;
    int32_t* status;
    Header* headers;
    void* parts;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes to shared memory, zeros where `bytes` is 0 (the source is then not read).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x cut off after its first 8 bits: a bf16 value.
__device__ __forceinline__ float top16(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

// The arithmetic on a tile of KT keys and values, by one warp.  The tile's row r begins at r * ROWB
// and its 16-byte piece c lies in place c ^ (r & 7), so that reads of one piece of 8 rows, and of
// one whole row, touch every bank once.

// Where dimension e of row r lies among a warp's sums: 8 lanes of neighbouring dimensions and 4 rows
// of even number write to 32 banks.
__device__ __forceinline__ int put_place(int D, int r, int e) {
    return r * D + (e ^ ((r >> 1 & 3) << 3));
}

// HEADS_ = 2: the rows of two neighbouring kv heads, next to one another in memory, are one row of D
// dimensions (and the two one head for the dealing).  Every head has its own query rows, maxima and
// sums; its scores take its half of a key's row, and its outputs its half of a value's.
template <int D_, int NQ, int HEADS_ = 1>
struct Bf16Math {
    using T = __nv_bfloat16;
    static constexpr int D = D_, ROWS = 8 * NQ, ROWB = D * 2, KT = HALF / ROWB;
    static constexpr int HEADS = HEADS_, DH = D / HEADS, MROWS = ROWS * HEADS;
    static constexpr int NI = NQ * HEADS, KH = DH / 16;    // tiles of scores; steps of a head's
    static constexpr int QROW = ROWB + 16;           // 16 more bytes: rows begin in other banks
    static constexpr int QBYTES = ROWS * QROW, SCRATCH = 0, NPASS = NQ;
    static constexpr bool BY_WARPS = false, SPARE = ROWS * D <= 1536;   // see ByWarps
    static constexpr int S = 3, BLOCKS = 2;          // stages of a warp's ring, blocks an SM

    // The queries' fragments stay in registers where these suffice; 24 rows of 128 would take 48 on
    // top of the sums' 96, and are read from shared memory for every 16 keys.
    static constexpr bool KEEP_Q = NQ * D <= 256;

    uint32_t qf[KEEP_Q ? NQ : 1][D / 16][2];
    float m[NI][2], l[NI][2], acc[NQ][D / 16][4];

    __device__ static __forceinline__ int q_place(int r, int c) { return r * QROW + c * 16; }

    __device__ __forceinline__ void begin(const unsigned char* qs, int lane) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                if (KEEP_Q) {
                    const unsigned char* at =
                        qs + (8 * i + lane / 4) * QROW + 32 * k + 4 * (lane & 3);
                    qf[i][k][0] = *reinterpret_cast<const uint32_t*>(at);
                    qf[i][k][1] = *reinterpret_cast<const uint32_t*>(at + 16);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][k][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            m[i][0] = m[i][1] = -INFINITY;
            l[i][0] = l[i][1] = 0.f;
        }
    }

    // Bit r of `ok`: key r counts.
    __device__ __forceinline__ void tile(const unsigned char* ks, const unsigned char* vs,
                                         const unsigned char* qs, unsigned char*, unsigned ok,
                                         float scale, int lane) {
        const uint32_t kb = sm100::smem_u32(ks), vb = sm100::smem_u32(vs);
        // lanes of a ldmatrix: query row lane % 8, pieces of 8 dimensions lane / 8
        const uint32_t qb = sm100::smem_u32(qs) + (lane & 7) * QROW + (lane >> 3) * 16;
#pragma unroll
        for (int j = 0; j < KT; j += 16) {
            float s[NI][4];                      // tile i: head i / NQ, query rows 8 (i % NQ) on
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
                uint32_t a[2][4];
                const int r = j + (lane & 15), c = 2 * k + (lane >> 4);
                ldmatrix4(a[0], kb + r * ROWB + ((c ^ (r & 7)) << 4));
                ldmatrix4(a[1], kb + r * ROWB + (((c + 2) ^ (r & 7)) << 4));
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    uint32_t b[4];
                    if (KEEP_Q) {
                        b[0] = qf[i][k][0];
                        b[1] = qf[i][k][1];
                        b[2] = qf[i][k + 1][0];
                        b[3] = qf[i][k + 1][1];
                    } else {
                        ldmatrix4(b, qb + 8 * i * QROW + 32 * k);
                    }
                    mma_16x8x16(s[k / KH * NQ + i], a[0], b[0], b[1]);
                    mma_16x8x16(s[k / KH * NQ + i], a[1], b[2], b[3]);
                }
            }
            // s[i]: key lane/4 (0, 1) and lane/4 + 8 (2, 3), queries 2 (lane & 3) and the next
            const bool ok0 = ok >> (j + lane / 4) & 1, ok1 = ok >> (j + 8 + lane / 4) & 1;
            uint32_t w[3][NI][2];
            bool up = false;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[i][e] = ok0 ? s[i][e] * scale : -INFINITY;
                    s[i][2 + e] = ok1 ? s[i][2 + e] * scale : -INFINITY;
                    up |= s[i][e] > m[i][e] || s[i][2 + e] > m[i][e];
                }
            // the maxima rise ever more seldom: the lanes compare theirs only where one does
            if (__any_sync(~0u, up)) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(m[i][e], fmaxf(s[i][e], s[i][2 + e]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
                        // m = -inf: nothing summed up so far, whatever the factor
                        f[e] = m[i][e] == -INFINITY ? 0.f : ex2(m[i][e] - x);
                        l[i][e] *= f[e];
                        m[i][e] = x;
                    }
#pragma unroll
                    for (int k = 0; k < KH; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i % NQ][i / NQ * KH + k][e] *= f[e & 1];
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float part[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float base = m[i][e & 1] == -INFINITY ? 0.f : m[i][e & 1];
                    const float p = ex2(s[i][e] - base);
                    l[i][e & 1] += p;
                    part[0][e] = top16(p);
                    const float rest = p - part[0][e];
                    // no part of a weight above 0 is 0: 0 times an infinite value would be NaN
                    const float least = fmaf(p, 0x1p-30f, fminf(p, 0x1p-133f));
                    part[1][e] = fmaxf(top16(rest), least);
                    part[2][e] = fmaxf(rest - top16(rest), least);
                }
#pragma unroll
                for (int t = 0; t < 3; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        w[t][i][e] = transpose8x8(
                            __byte_perm(__float_as_uint(part[t][2 * e]),
                                        __float_as_uint(part[t][2 * e + 1]), 0x7632));
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                const int r = j + (lane & 7) + (lane >> 4) * 8, c = 2 * k + (lane >> 3 & 1);
                ldmatrix4_trans(a, vb + r * ROWB + ((c ^ (r & 7)) << 4));
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const int h = k / KH * NQ + i;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};     // of these 16 keys, the least parts first
#pragma unroll
                    for (int t = 2; t >= 0; --t) mma_16x8x16(sum, a, w[t][h][0], w[t][h][1]);
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 x = sm100::add2(make_float2(acc[i][k][e], acc[i][k][e + 1]),
                                                     make_float2(sum[e], sum[e + 1]));
                        acc[i][k][e] = x.x;
                        acc[i][k][e + 1] = x.y;
                    }
                }
            }
        }
    }

    // The warp's maxima and sums of all rows, head after head.
    __device__ __forceinline__ void end(float* wm, float* wl, int lane) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(~0u, l[i][e], o);
                if (lane < 4) {
                    wm[8 * i + 2 * lane + e] = m[i][e];
                    wl[8 * i + 2 * lane + e] = l[i][e];
                }
            }
    }

    // The sums of 8 rows of values, each in put_place's order.
    __device__ __forceinline__ void put(int pass, float* to, int lane) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
            if (i == pass)
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[put_place(D, 2 * (lane & 3) + (e & 1),
                                     16 * k + lane / 4 + (e >> 1) * 8)] = acc[i][k][e];
    }
};

template <int D_, int R>
struct F32Math {
    using T = float;
    static constexpr int D = D_, ROWS = R, ROWB = D * 4, KT = HALF / ROWB;
    static constexpr int HEADS = 1, DH = D, MROWS = R;
    static constexpr int CPR = ROWB / 16, KI = 32 / CPR;   // pieces a row; rows a warp-wide read
    // a query row in parts of 32 dimensions, 16 bytes between them: the parts begin in other banks
    static constexpr int QROW = D / 32 * 144;
    static constexpr int QBYTES = R * QROW, SCRATCH = KT * R * 4, NPASS = 1;
    static constexpr bool BY_WARPS = false, SPARE = R * D <= 1024;
    // Three blocks an SM with a tile less each, where latency of the arithmetic bounds the kernel and
    // 168 registers do (8 rows of 128: 104 -> 98 us; 12 rows, with them spilled, 284 -> 327).
    static constexpr bool MORE = R == 8 && D == 128;
    static constexpr int S = MORE ? 2 : 3, BLOCKS = MORE ? 3 : 2;

    float m[R], l[R];
    float2 acc[R][2];            // dimensions 4 (lane % CPR) and on

    __device__ static __forceinline__ int q_place(int r, int c) {
        return r * QROW + c / 8 * 144 + c % 8 * 16;
    }

    __device__ __forceinline__ void begin(const unsigned char*, int) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            acc[r][0] = acc[r][1] = make_float2(0.f, 0.f);
        }
    }

    __device__ __forceinline__ void tile(const unsigned char* ks, const unsigned char* vs,
                                         const unsigned char* qs, unsigned char* scratch,
                                         unsigned ok, float scale, int lane) {
        const int key = lane % KT, part = lane / KT;       // this lane's 32 of the D dimensions
        float2 s2[R];                                      // even and odd dimensions
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) s2[r] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 k = *reinterpret_cast<const float4*>(
                ks + key * ROWB + (((part * 8 + c) ^ (key & 7)) << 4));
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q =
                    *reinterpret_cast<const float4*>(qs + r * QROW + part * 144 + c * 16);
                s2[r] = sm100::fma2(make_float2(q.x, q.y), make_float2(k.x, k.y), s2[r]);
                s2[r] = sm100::fma2(make_float2(q.z, q.w), make_float2(k.z, k.w), s2[r]);
            }
        }
        const bool okk = ok >> key & 1;
        bool up = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = s2[r].x + s2[r].y;
#pragma unroll
            for (int o = KT; o < 32; o <<= 1) s[r] += __shfl_xor_sync(~0u, s[r], o);
            s[r] = okk ? s[r] * scale : -INFINITY;
            up |= s[r] > m[r];
        }
        if (__any_sync(~0u, up)) {             // as for bf16
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float x = fmaxf(m[r], s[r]);
#pragma unroll
                for (int o = 1; o < KT; o <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
                const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - x);
                l[r] *= f;
                m[r] = x;
                acc[r][0] = sm100::mul2(acc[r][0], make_float2(f, f));
                acc[r][1] = sm100::mul2(acc[r][1], make_float2(f, f));
            }
        }
        float* pk = reinterpret_cast<float*>(scratch);     // [KT][R]
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = ex2(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
            l[r] += s[r];
        }
        if (part == 0)
#pragma unroll
            for (int r = 0; r < R; r += 4)
                *reinterpret_cast<float4*>(pk + key * R + r) =
                    make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
        __syncwarp();
        const int c = lane % CPR;
#pragma unroll
        for (int j = 0; j < KT; j += KI) {
            const int row = j + lane / CPR;
            const float4 v =
                *reinterpret_cast<const float4*>(vs + row * ROWB + ((c ^ (row & 7)) << 4));
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 p = *reinterpret_cast<const float4*>(pk + row * R + r);
                const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 pp = make_float2(pr[e], pr[e]);
                    acc[r + e][0] = sm100::fma2(pp, make_float2(v.x, v.y), acc[r + e][0]);
                    acc[r + e][1] = sm100::fma2(pp, make_float2(v.z, v.w), acc[r + e][1]);
                }
            }
        }
    }

    __device__ __forceinline__ void end(float* wm, float* wl, int lane) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int o = 1; o < KT; o <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], o);
            if (lane == 0) {
                wm[r] = m[r];
                wl[r] = l[r];
            }
        }
    }

    __device__ __forceinline__ void put(int, float* to, int lane) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x[4] = {acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y};
            if (KI == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += __shfl_xor_sync(~0u, x[e], 16);
            if (lane < CPR)
                *reinterpret_cast<float4*>(to + put_place(D, r, 4 * lane)) =
                    make_float4(x[0], x[1], x[2], x[3]);
        }
    }
};

// The same with short pairs worked on by single warps.  A block takes 1.5 us and more to end a pair,
// and one warp little longer for a short one altogether, while the block's others do as much: 187 x
// 16 pairs of 2 keys 28 -> 14 us, 192 x 16 of 70 keys of 64 dimensions 28 -> 22.  A kernel of its
// own, for batches that may have enough such pairs: others would be 3 to 6 % slower for the code
// that they have no use for.  Not where the rows' sums leave no registers to spare (SPARE): there
// the kernel would be 9 % slower on batches that are long after all.
template <class M>
struct ByWarps : M {
    static constexpr bool BY_WARPS = true;
    static constexpr int S = 3, BLOCKS = 2;
    static_assert(M::QBYTES <= STAGE, "a stage of the ring holds the queries");
};

// Keys [first, len) of sequence b.
__device__ __forceinline__ void key_range(const Params& p, int b, uint32_t& first, uint32_t& len) {
    const int64_t cap = (int64_t)p.table.max_pages << p.pool.page_shift;
    const int n = p.lens[b];
    len = n;
    if (n < 0 || n > cap) {
        paged_flag(p.status, GRET_PAGED_BAD_LENGTH);
        len = n < 0 ? 0 : (uint32_t)cap;
    }
    first = p.window > 0 && len > (uint32_t)p.window ? len - p.window : 0;
}

__device__ __forceinline__ int units_between(uint32_t first, uint32_t len) {
    return (int)((len - first + UNIT - 1) / UNIT);
}

__device__ __forceinline__ int units_of(const Params& p, int b) {
    uint32_t first, len;
    key_range(p, b, first, len);
    return units_between(first, len);
}

// What ending a pair costs, in units: 1.5 us, and 1.2 for each 8 rows more, when a block reads 22 KB
// a us.
template <class M>
constexpr int end_units() {
    constexpr int unit_ns = UNIT * 2 * M::ROWB * M::BLOCKS / 44, end_ns = 300 + 1200 * M::NPASS;
    return (end_ns + unit_ns / 2) / unit_ns < 1 ? 1 : (end_ns + unit_ns / 2) / unit_ns;
}

// The sequences that a walk over the batch stops at.
enum Kind : int { ANY, LONG, SHORT };

template <class M>
__device__ __forceinline__ bool is_short(uint32_t first, uint32_t len) {
    return M::BY_WARPS && len - first <= SHORT_TILES * M::KT;
}

// A stretch of one pair's units that a block works on: units [t0, t1) of the nu that hold keys;
// end_units() units for the pair's end follow those in the count.
template <class M>
struct Segment {
    static constexpr int LAST = end_units<M>();

    int64_t u;                   // of all units of this kind, the one t0 stands for
    uint32_t first, len;
    int b, pr, nu, t0, t1;

    // At unit u, in sequence b_, whose units begin at b_unit, of those dealt up to u1; false if
    // there are no keys in [u, u1).
    __device__ __forceinline__ bool start(const Params& p, Kind kind, int b_, int64_t b_unit,
                                          int64_t u_, int64_t u1) {
        b = b_;
        u = u_;
        key_range(p, b, first, len);
        nu = units_between(first, len);
        const int64_t x = u - b_unit;             // = pr (nu + LAST) + t0
        if (x <= INT_MAX) {                       // a fifth of the time of a division in 64 bits
            pr = (int)x / (nu + LAST);
            t0 = (int)x % (nu + LAST);
        } else {
            pr = (int)(x / (nu + LAST));
            t0 = (int)(x % (nu + LAST));
        }
        t1 = (int)min((int64_t)nu, t0 + (u1 - u));
        // short pairs belong whole to the warp that their first unit is dealt to; a range may also
        // begin among the units of an end
        if (t0 >= (kind == SHORT ? 1 : nu)) return next(p, kind, u1);
        if (kind == SHORT) t1 = nu;
        return true;
    }
    __device__ __forceinline__ uint32_t key0() const { return first + (uint32_t)t0 * UNIT; }
    __device__ __forceinline__ uint32_t key1() const {
        return t1 == nu ? len : first + (uint32_t)t1 * UNIT;
    }
    // To the next one of a range that ends before u1.
    __device__ __forceinline__ bool next(const Params& p, Kind kind, int64_t u1) {
        u += nu + LAST - t0;
        if (u >= u1) return false;
        t0 = 0;                  // only a block's last segment ends inside its pair
        if (++pr == p.pool.H * p.QG) {
            pr = 0;
            do {
                if (++b == p.table.S) return false;
                key_range(p, b, first, len);
            } while (len == first || (kind != ANY && (kind == SHORT) != is_short<M>(first, len)));
            nu = units_between(first, len);
        }
        t1 = kind == SHORT ? nu : (int)min((int64_t)nu, u1 - u);
        return true;
    }
    // Its queries: the first of them, and how many (of each of its heads, G further on).
    __device__ __forceinline__ int64_t head(const Params& p) const {
        return (int64_t)b * p.Hq + pr / p.QG * (M::HEADS * p.G) + pr % p.QG * M::ROWS;
    }
    __device__ __forceinline__ int rows(const Params& p) const {
        return min(M::ROWS, p.G - pr % p.QG * M::ROWS);
    }
};

// How U units are dealt to n workers: worker c has units [begin(c), begin(c + 1)), each of the first
// `more` one more than the others' `each`.  With fewer units than workers, the first U take one
// each: a pair's parts lie in consecutive blocks.  A pair counts for more units than its keys fill,
// since ending one (joining the warps' parts, writing the outcome) takes time too: counted by keys
// alone, blocks of many pairs came last.
struct Deal {
    int64_t U, each;
    int more;

    Deal() = default;
    __device__ __forceinline__ Deal(int64_t units, int n)
        : U(units), each(units / n), more((int)(units % n)) {}
    __device__ __forceinline__ int64_t begin(int c) const { return each * c + min(c, more); }
    // The worker that holds unit x.
    __device__ __forceinline__ int worker_of(int64_t x) const {
        const int64_t head = (each + 1) * more;
        return x < head ? (int)(x / (each + 1)) : more + (int)((x - head) / each);
    }
};

// Units that sequence b is dealt as: of each pair its keys' and those of its end.
template <class M>
__device__ __forceinline__ int64_t dealt_units(const Params& p, int b, bool& shorts) {
    uint32_t first, len;
    key_range(p, b, first, len);
    shorts = len > first && is_short<M>(first, len);
    return len == first ? 0
                        : (int64_t)(units_between(first, len) + end_units<M>()) * (p.pool.H * p.QG);
}

struct DealSmem {
    int64_t longs[NW], shorts[NW], unit[NW + 1];
    int n_short[NW], b[NW + 1];
};

template <class M>
using PartOf = Part<M::MROWS, M::ROWS, M::D>;

// What is dealt to a block and to this warp of it: units of long pairs and of short ones, the
// sequence of the first of them, and that one's first unit.
struct Share {
    Deal longs, shorts;
    int long_b, short_b;         // -1: none
    int64_t long_b_unit, short_b_unit;
    Kind kind;                   // of the pairs dealt to blocks: LONG, or ANY where all are
};

// Inclusive sum of x over the warp's lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

template <class M>
__device__ __forceinline__ Share share_of(const Params& p, DealSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    const int B = p.table.S, pairs_b = p.pool.H * p.QG, per = (B + NT - 1) / NT;
    const int b0 = tid * per, b1 = min(B, b0 + per);
    // short pairs go to warps where there are enough to go round, else to blocks like the others
    bool by_warps = M::BY_WARPS;
    int64_t longs = 0, shorts = 0;                // units of this thread's sequences
    int n_short = 0;
    for (int i = b0; i < b1; ++i) {
        bool is;
        const int64_t x = dealt_units<M>(p, i, is);
        is &= by_warps;
        longs += is ? 0 : x;
        shorts += is ? x : 0;
        n_short += is;
    }
    const int64_t longs_upto = warp_scan(longs);
    if (lane == 31) sm.longs[warp] = longs_upto;
    int64_t shorts_upto = 0;
    if (by_warps) {
        shorts_upto = warp_scan(shorts);
        n_short = __reduce_add_sync(~0u, n_short);
        if (lane == 31) {
            sm.shorts[warp] = shorts_upto;
            sm.n_short[warp] = n_short;
        }
    }
    __syncthreads();
    int64_t longs_before = longs_upto - longs, longs_all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) longs_before += sm.longs[w];
        longs_all += sm.longs[w];
    }
    int64_t shorts_before = shorts_upto - shorts, shorts_all = 0;
    if (by_warps) {
        n_short = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) shorts_before += sm.shorts[w];
            shorts_all += sm.shorts[w];
            n_short += sm.n_short[w];
        }
        by_warps = (int64_t)n_short * pairs_b >= MIN_SHORT;
        if (!by_warps) {
            longs += shorts;
            longs_before += shorts_before;
            longs_all += shorts_all;
            shorts_all = 0;
        }
    }
    Share r = {Deal(longs_all, 148 * M::BLOCKS), Deal(shorts_all, 148 * M::BLOCKS * NW), -1, -1, 0, 0,
               by_warps ? LONG : ANY};
    // the thread that holds the first unit of a share says where it is
    auto find = [&](int64_t u, int64_t at, int64_t mine, bool want, int slot) {
        if (u < at || u >= at + mine) return;
        for (int i = b0; i < b1; ++i) {
            bool is;
            const int64_t x = per == 1 ? mine : dealt_units<M>(p, i, is);
            if (per > 1 && by_warps && is != want) continue;
            if (u < at + x) {
                sm.b[slot] = i;
                sm.unit[slot] = at;
                return;
            }
            at += x;
        }
    };
    if (c < longs_all) find(r.longs.begin(c), longs_before, longs, false, NW);
    if (by_warps)
#pragma unroll 1
        for (int w = 0; w < NW; ++w)
            if (c * NW + w < shorts_all)
                find(r.shorts.begin(c * NW + w), shorts_before, shorts, true, w);
    __syncthreads();
    if (c < longs_all) {
        r.long_b = sm.b[NW];
        r.long_b_unit = sm.unit[NW];
    }
    if (c * NW + warp < shorts_all) {
        r.short_b = sm.b[warp];
        r.short_b_unit = sm.unit[warp];
    }
    return r;
}

// A warp's walk over the tiles that it is to load.  A tile's page-table entries are read when it
// enters the queue `ahead`, S - 1 tiles before they are needed: one latency for all of a ring's first
// tiles.
template <class M>
struct Loader {
    static constexpr int KT = M::KT, ROWB = M::ROWB, CPR = ROWB / 16, S = M::S;

    struct Tile {
        int64_t head;            // bytes from a slot to its head's row
        uint32_t at, end;        // its first key, and the end of its segment (at >= end: no tile)
        int id;                  // of lane's key: its page
    };

    Tile ahead[S - 1] = {};
    Segment<M> seg;
    int64_t u1;
    uint32_t at, end, skip, step;   // this warp's first tile of a segment, and from one to the next
    Kind kind;
    bool more;

    __device__ __forceinline__ Loader(const Params& p, const Segment<M>& first, Kind k,
                                      int64_t end_unit, uint32_t skip_, uint32_t step_, int lane)
        : seg(first), u1(end_unit), at(first.key0() + skip_), end(first.key1()), skip(skip_),
          step(step_), kind(k), more(true) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) look_up(p, ahead[i], lane);
    }

    __device__ __forceinline__ void look_up(const Params& p, Tile& t, int lane) {
        while (more && at >= end) {
            more = seg.next(p, kind, u1);
            at = seg.key0() + skip;
            end = seg.key1();
        }
        t.at = at;
        t.end = more ? end : 0;
        t.head = seg.pr / p.QG * p.pool.sh;
        t.id = -1;
        if (lane < KT && at + lane < t.end)
            t.id = p.table.entries[seg.b * p.table.stride + ((at + lane) >> p.pool.page_shift)];
        at += step;
    }

    // Load the first tile of the queue, and take up another: a bit for every key that counts.
    __device__ __forceinline__ unsigned load(const Params& p, unsigned char* stage, int lane) {
        const Tile t = ahead[0];
        unsigned ok = 0;
        if (t.at < t.end) {
            const bool in = lane < KT && t.at + lane < t.end;
            const bool good = in && (unsigned)t.id < (unsigned)p.pool.n_pages;
            if (in && !good) paged_flag(p.status, GRET_PAGED_BAD_PAGE);
            ok = __ballot_sync(~0u, good);
            const int64_t off =
                good ? t.id * p.pool.sp +
                           ((t.at + lane) & ((1u << p.pool.page_shift) - 1)) * p.pool.st + t.head
                     : 0;
#pragma unroll
            for (int i = 0; i < S - 2; ++i) ahead[i] = ahead[i + 1];
            look_up(p, ahead[S - 2], lane);
            const uint32_t to = sm100::smem_u32(stage);
            const int c = lane % CPR;
#pragma unroll
            for (int i = 0; i < KT * CPR / 32; ++i) {
                const int r = i * (32 / CPR) + lane / CPR;
                const int64_t o = __shfl_sync(~0u, off, r) + c * 16;
                const uint32_t dst = to + r * ROWB + ((c ^ (r & 7)) << 4);
                const uint32_t bytes = ok >> r & 1 ? 16 : 0;
                cp_async_16_or_zero(dst, p.pool.k + o, bytes);
                cp_async_16_or_zero(dst + HALF, p.pool.v + o, bytes);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return ok;
    }
};

// Of piece c of row r of the queries (and outputs) from `head` on: its place among all queries' pieces.
template <class M>
__device__ __forceinline__ int64_t query_piece(const Params& p, int64_t head, int r, int c) {
    constexpr int PIECES = M::ROWB / 16 / M::HEADS;        // of a head's row
    return (head + (M::HEADS == 1 ? 0 : c / PIECES * p.G) + r) * PIECES + c % PIECES;
}

// Where in a row's D dimensions e lies: the row of its maximum and sum.
template <class M>
__device__ __forceinline__ int max_row(int row, int e) {
    return M::HEADS == 1 ? row : e / M::DH * M::ROWS + row;
}

// Four dimensions of row r of the outputs from `head` on, and the row's lse from maximum (log2) and
// sum.
template <class M>
__device__ __forceinline__ void put_out(const Params& p, int64_t head, int r, int e,
                                        const float (&a)[4], float mx, float z) {
    using T = typename M::T;
    const int64_t row = head + (M::HEADS == 1 ? 0 : e / M::DH * p.G) + r;
    T* o = static_cast<T*>(p.o) + row * M::DH + e % M::DH;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = from_f32<T>(a[x] / z);
    if (p.lse && e % M::DH == 0) p.lse[row] = (mx + log2f(z)) * LN2;
}

// The short pairs dealt to this warp, one after another, each from its first key to its output.  Two
// stages of the ring hold tiles, the third the queries.
template <class M>
__device__ __forceinline__ void work_by_warp(const Params& p, M& math, const Share& share,
                                             unsigned char* ring, unsigned char* scratch, float* wm,
                                             float* wl) {
    constexpr int D = M::D, CPR = M::ROWB / 16;
    constexpr int PR = M::ROWS / M::NPASS, FIT = STAGE / (PR * D * 4);
    const int lane = threadIdx.x & 31, worker = blockIdx.x * NW + (threadIdx.x >> 5);
    const int64_t u1 = share.shorts.begin(worker + 1);
    Segment<M> seg;
    if (share.short_b < 0 || !seg.start(p, SHORT, share.short_b, share.short_b_unit,
                                        share.shorts.begin(worker), u1))
        return;
    unsigned char* qs = ring + 2 * STAGE;
    Loader<M> loader(p, seg, SHORT, u1, 0, M::KT, lane);
    unsigned ok = loader.load(p, ring, lane);
    int stage = 0;
    for (bool go = true; go;) {
        const int rows = seg.rows(p);
        const int64_t head = seg.head(p);
        const uint4* q = static_cast<const uint4*>(p.q);
        for (int x = lane; x < M::ROWS * CPR; x += 32)
            cp_async_16_or_zero(
                sm100::smem_u32(qs + M::q_place(x / CPR, x % CPR)),
                x < rows * CPR ? q + query_piece<M>(p, head, x / CPR, x % CPR) : q,
                x < rows * CPR ? 16 : 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const uint32_t key0 = seg.key0(), key1 = seg.key1();
        for (uint32_t k = key0; k < key1; k += M::KT) {
            const unsigned ok_next = loader.load(p, ring + (stage ^ 1) * STAGE, lane);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            if (k == key0) math.begin(qs, lane);
            const unsigned char* t = ring + stage * STAGE;
            math.tile(t, t + HALF, qs, scratch, ok, p.scale_log2, lane);
            __syncwarp();
            ok = ok_next;
            stage ^= 1;
        }
        math.end(wm, wl, lane);
        // the tile last worked on has made room
        float* buf = reinterpret_cast<float*>(ring + (stage ^ 1) * STAGE);
#pragma unroll 1
        for (int pass = 0; pass < M::NPASS; pass += FIT) {
            for (int i = 0; i < FIT && pass + i < M::NPASS; ++i)
                math.put(pass + i, buf + i * PR * D, lane);
            __syncwarp();
            const int row0 = pass * PR, n = min(rows - row0, FIT * PR);
            for (int i = lane; i < n * (D / 4); i += 32) {
                const int r = i / (D / 4), e = i % (D / 4) * 4;
                const float4 x = *reinterpret_cast<const float4*>(buf + put_place(D, r, e));
                const float a[4] = {x.x, x.y, x.z, x.w};
                put_out<M>(p, head, row0 + r, e, a, wm[max_row<M>(row0 + r, e)],
                           wl[max_row<M>(row0 + r, e)]);
            }
            __syncwarp();
        }
        go = seg.next(p, SHORT, u1);
    }
}

template <class M>
__global__ void __launch_bounds__(NT, M::BLOCKS) paged_attn_kernel(const Params p) {
    constexpr int D = M::D, KT = M::KT, CPR = M::ROWB / 16, S = M::S, RING = S * STAGE;
    constexpr int QC = (M::ROWS * CPR + NT - 1) / NT;      // pieces of the queries a thread moves
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float wm[NW][M::MROWS], wl[NW][M::MROWS];
    __shared__ const float* wput[NW];
    __shared__ DealSmem deal_smem;
    __shared__ Deal longs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    unsigned char* ring = smem + warp * RING;
    unsigned char* qs = smem + NW * RING;
    unsigned char* scratch = qs + M::QBYTES + warp * M::SCRATCH;
    wait_for_previous();
    let_next_start();
    const Share share = share_of<M>(p, deal_smem);
    if (tid == 0) {
        p.headers[c] = {0, 0, 0};
        longs = share.longs;
    }
    M math;
    if (M::BY_WARPS && share.kind == LONG) {
        work_by_warp<M>(p, math, share, ring, scratch, wm[warp], wl[warp]);
        __syncthreads();
    }
    const int64_t u1 = share.longs.begin(c + 1);
    Segment<M> seg;
    if (share.long_b < 0 || !seg.start(p, share.kind, share.long_b, share.long_b_unit,
                                       share.longs.begin(c), u1))
        return;

    // A segment's queries: read one segment ahead, put into shared memory when it begins.
    uint4 qn[QC];
    auto read_q = [&](const Segment<M>& s) {
        const uint4* q = static_cast<const uint4*>(p.q);
        const int64_t head = s.head(p);
        const int n = s.rows(p) * CPR;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const int x = tid + i * NT;
            qn[i] = x < n ? q[query_piece<M>(p, head, x / CPR, x % CPR)] : make_uint4(0, 0, 0, 0);
        }
    };
    auto put_q = [&]() {
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const int x = tid + i * NT;
            if (x < M::ROWS * CPR)
                *reinterpret_cast<uint4*>(qs + M::q_place(x / CPR, x % CPR)) = qn[i];
        }
    };
    read_q(seg);
    Loader<M> loader(p, seg, share.kind, u1, warp * KT, NW * KT, lane);
    unsigned ok[S];
#pragma unroll
    for (int i = 0; i < S - 1; ++i) ok[i] = loader.load(p, ring + i * STAGE, lane);
    int stage = 0;
    put_q();
    __syncthreads();

    for (bool go = true; go;) {
        Segment<M> nx = seg;
        go = nx.next(p, share.kind, u1);
        if (go) read_q(nx);
        math.begin(qs, lane);
        const uint32_t key1 = seg.key1();
        for (uint32_t k = seg.key0() + warp * KT; k < key1; k += NW * KT) {
            ok[S - 1] = loader.load(p, ring + (stage == 0 ? S - 1 : stage - 1) * STAGE, lane);
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();
            const unsigned char* t = ring + stage * STAGE;
            math.tile(t, t + HALF, qs, scratch, ok[0], p.scale_log2, lane);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S - 1; ++i) ok[i] = ok[i + 1];
            stage = stage == S - 1 ? 0 : stage + 1;
        }
        // join the warps' parts, through the ring's one stage that no load is under way to
        const int rows = seg.rows(p);
        const int64_t head0 = seg.head(p);
        const bool whole = seg.t0 == 0 && seg.t1 == seg.nu;
        PartOf<M>* part = static_cast<PartOf<M>*>(p.parts) + 2 * c + (seg.t0 == 0);
        if (!whole && seg.t0 == 0 && tid == 0)
            p.headers[c] = {(int32_t)head0, (int16_t)rows,
                            (int16_t)(longs.worker_of(seg.u + seg.nu - 1) - c + 1)};
        // in passes of as many rows as the stage holds; when the block ends here, nothing is under
        // way, and one pass does
        constexpr int PR = M::ROWS / M::NPASS;             // rows of a tile of queries
        constexpr int FIT = STAGE / (PR * D * 4) < M::NPASS ? STAGE / (PR * D * 4) : M::NPASS;
        static_assert(M::ROWS * D * 4 <= RING && FIT >= 1, "");
        const int np = go ? FIT : M::NPASS;
        float* mine_put = reinterpret_cast<float*>(
            ring + (go ? (stage == 0 ? S - 1 : stage - 1) * STAGE : 0));
        if (lane == 0) wput[warp] = mine_put;
        math.end(wm[warp], wl[warp], lane);
#pragma unroll 1
        for (int pass = 0; pass < M::NPASS; pass += np) {
            for (int i = 0; i < np && pass + i < M::NPASS; ++i)
                math.put(pass + i, mine_put + i * PR * D, lane);
            __syncthreads();
            if (pass == 0 && go) put_q();
            const int row0 = pass * PR, n = min(rows - row0, np * PR);
            for (int i = tid; i < n * (D / 4); i += NT) {
                const int r = i / (D / 4), e = i % (D / 4) * 4, row = row0 + r;
                const int mr = max_row<M>(row, e);
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w) mx = fmaxf(mx, wm[w][mr]);
                const float base = mx == -INFINITY ? 0.f : mx;
                float a[4] = {}, z = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float f = ex2(wm[w][mr] - base);
                    const float4 x = *reinterpret_cast<const float4*>(wput[w] + put_place(D, r, e));
                    a[0] += x.x * f;
                    a[1] += x.y * f;
                    a[2] += x.z * f;
                    a[3] += x.w * f;
                    z += wl[w][mr] * f;
                }
                if (whole) {
                    put_out<M>(p, head0, row, e, a, mx, z);
                } else {
                    *reinterpret_cast<float4*>(&part->a[row][e]) =
                        make_float4(a[0], a[1], a[2], a[3]);
                    if (e % M::DH == 0) {
                        part->m[mr] = mx;
                        part->l[mr] = z;
                    }
                }
            }
            if (go) __syncthreads();
        }
        seg = nx;
    }
}

// Row r of the n parts, to row r of the outputs from `head` on: a warp a quarter of the parts, a lane
// D / 32 dimensions.  All that a row is made of is on its way before any of it is looked at, up to 32
// parts.
template <class M>
__device__ __forceinline__ void join_row(const Params& p, const PartOf<M>* parts, int n, int r,
                                         int64_t head) {
    using T = typename M::T;
    constexpr int D = M::D, E = D / 32, EH = E / M::HEADS, UN = 8, GRID = 148 * M::BLOCKS;
    constexpr int PER = (GRID + NT - 1) / NT, H = M::HEADS;
    __shared__ float w[H][GRID];                           // the parts' weights
    __shared__ float sums[NW][D], red[2][H][NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // part k: the tail of block c, then the heads of those that follow
    float x[UN][E], m[H][PER], l[H][PER];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int k = k0 + i * NW;
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[i][e] = k < n ? parts[2 * k + (k == 0)].a[r][lane + 32 * e] : 0.f;
        }
    };
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int k = tid + i * NT;
            m[h][i] = k < n ? parts[2 * k + (k == 0)].m[h * M::ROWS + r] : -INFINITY;
            l[h][i] = k < n ? parts[2 * k + (k == 0)].l[h * M::ROWS + r] : 0.f;
        }
    fetch(warp);
    float mx[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        mx[h] = m[h][0];
#pragma unroll
        for (int i = 1; i < PER; ++i) mx[h] = fmaxf(mx[h], m[h][i]);
        for (int o = 16; o; o >>= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], o));
        if (lane == 0) red[0][h][warp] = mx[h];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < NW; ++i) mx[h] = fmaxf(mx[h], red[0][h][i]);
        const float base = mx[h] == -INFINITY ? 0.f : mx[h];
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float f = ex2(m[h][i] - base);
            if (tid + i * NT < n) w[h][tid + i * NT] = f;
            z += f * l[h][i];
        }
        for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
        if (lane == 0) red[1][h][warp] = z;
    }
    __syncthreads();
    float a[E] = {};
    for (int k0 = warp; k0 < n; k0 += NW * UN) {
        if (k0 != warp) fetch(k0);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int k = k0 + i * NW;
            float f[H];
#pragma unroll
            for (int h = 0; h < H; ++h) f[h] = k < n ? w[h][k] : 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = fmaf(f[e / EH], x[i][e], a[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][lane + 32 * e] = a[e];
    __syncthreads();
    if (tid < D) {
        const int h = tid / M::DH;
        float y = 0.f, z = 0.f, top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            y += sums[i][tid];
            z += red[1][h][i];
            top = fmaxf(top, red[0][h][i]);
        }
        const int64_t row = head + (H == 1 ? 0 : h * p.G) + r;
        static_cast<T*>(p.o)[row * M::DH + tid % M::DH] = from_f32<T>(y / z);
        if (p.lse && tid % M::DH == 0) p.lse[row] = (top + log2f(z)) * LN2;
    }
}

// Blocks (c, y) join the parts of the pair that block c of the kernel above began and did not
// finish, each every JOIN_Y-th row of it.
template <class M>
__global__ void __launch_bounds__(NT) paged_join_kernel(const Params p) {
    using T = typename M::T;
    constexpr int DH = M::DH;
    const int tid = threadIdx.x, c = blockIdx.x;
    wait_for_previous();
    const Header h = p.headers[c];
    for (int r = blockIdx.y; r < h.rows; r += gridDim.y) {
        __syncthreads();
        join_row<M>(p, static_cast<const PartOf<M>*>(p.parts) + 2 * c, h.parts, r, h.head);
    }
    // sequences without keys: zeros
    for (int b = c; b < p.table.S; b += 148 * M::BLOCKS)
        if (units_of(p, b) == 0)
            for (int i = blockIdx.y; i < p.Hq; i += gridDim.y) {
                for (int e = tid; e < DH; e += NT)
                    static_cast<T*>(p.o)[((int64_t)b * p.Hq + i) * DH + e] = from_f32<T>(0.f);
                if (p.lse && tid == 0) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
            }
}

template <class M>
cudaError_t launch_form(const Params& p, cudaStream_t stream) {
    constexpr int grid = 148 * M::BLOCKS;
    constexpr int smem = NW * (M::S * STAGE + M::SCRATCH) + M::QBYTES;
    static_assert(M::BLOCKS * (smem + 3072) <= 228 * 1024 && grid <= MAX_GRID, "");
    cudaError_t e = allow_smem<paged_attn_kernel<M>>(smem, smem);
    if (e != cudaSuccess) return e;
    e = launch_early(paged_attn_kernel<M>, dim3(grid), NT, smem, stream, p);
    if (e != cudaSuccess) return e;
    return launch_early(paged_join_kernel<M>, dim3(grid, p.G < JOIN_Y ? p.G : JOIN_Y), NT, 0, stream,
                        p);
}

template <class M>
cudaError_t launch(Params& p, cudaStream_t stream) {
    p.QG = (p.G + M::ROWS - 1) / M::ROWS;
    using W = typename std::conditional<M::SPARE, ByWarps<M>, M>::type;
    return (int64_t)p.table.S * p.pool.H * p.QG >= MIN_SHORT ? launch_form<W>(p, stream)
                                                             : launch_form<M>(p, stream);
}

// Query rows a block works on at a time: all G heads of a group where they fit, else the fewest
// equal passes over the keys (each pass reads them again), in steps of 8 rows for bf16 and 4 for
// fp32.
int rows_of(bool bf16, int G) {
    const int most = bf16 ? MAXROWS_BF16 : MAXROWS_F32, step = bf16 ? 8 : 4;
    const int passes = (G + most - 1) / most, rows = (G + passes - 1) / passes;
    return (rows + step - 1) / step * step;
}

// Whether two heads of 64 dimensions can be worked on as one row of 128, where a group's query rows
// are one tile: they lie next to one another (see Bf16Math).  A key of one such head is a piece of 128
// bytes, which HBM serves at 0.84 of the rate of a plain copy: 32 sequences of 50000 tokens, 8 such
// heads, 587 us one by one and 479 two by two.
bool two_heads(bool bf16, int d, int G, const PagedPool& pool) {
    return bf16 && d == 64 && G <= 8 && pool.H % 2 == 0 && pool.sh == 128;
}

template <int D>
cudaError_t launch_d(bool bf16, int rows, Params& p, cudaStream_t stream) {
    if (bf16) switch (rows) {
        case 8: return launch<Bf16Math<D, 1>>(p, stream);
        case 16: return launch<Bf16Math<D, 2>>(p, stream);
        default: return launch<Bf16Math<D, 3>>(p, stream);
    }
    switch (rows) {
        case 4: return launch<F32Math<D, 4>>(p, stream);
        case 8: return launch<F32Math<D, 8>>(p, stream);
        case 12: return launch<F32Math<D, 12>>(p, stream);
        default: return launch<F32Math<D, 16>>(p, stream);
    }
}

}  // namespace

size_t paged_attn_workspace(bool bf16, int Hq, int Hkv, int d) {
    const size_t head = (MAX_GRID * sizeof(Header) + 255) / 256 * 256;
    const int G = Hq / Hkv, heads = bf16 && d == 64 && G <= 8 ? 2 : 1;   // whatever the strides
    return head + (size_t)2 * MAX_GRID * rows_of(bf16, G) * heads * (d + 2) * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
    Params p;
    p.q = a.q;
    p.lens = a.seq_lens;
    p.table = a.table;
    p.pool = a.pool;
    p.scale_log2 = a.scale * LOG2E;
    p.window = a.window;
    p.Hq = a.Hq;
    p.G = a.Hq / a.pool.H;
    p.o = a.o;
    p.lse = a.lse;
    p.status = a.status;
    p.headers = static_cast<Header*>(a.workspace);
    p.parts = static_cast<unsigned char*>(a.workspace) + (MAX_GRID * sizeof(Header) + 255) / 256 * 256;
    if (two_heads(a.bf16, a.d, p.G, a.pool)) {
        p.pool.H /= 2;
        p.pool.sh *= 2;
        return launch<Bf16Math<128, 1, 2>>(p, stream);
    }
    const int rows = rows_of(a.bf16, p.G);
    return a.d == 64 ? launch_d<64>(a.bf16, rows, p, stream)
                     : launch_d<128>(a.bf16, rows, p, stream);
}

}  // namespace gret
