// Attention over the 8-bit paged cache, split along the tokens: decode, verify and short extensions.
//
// The work is one pass over the cached keys and values, two bytes per (token, head dimension), for few
// query rows, so HBM bandwidth bounds it.  Steps of 32 tokens of all (request, key/value head, block of rows)
// items form one list, cut into equal pieces, one per warp, so that any mix of lengths fills the SMs; an item
// counts kItemSteps steps more than it has, for what beginning and ending it costs.  Warps work alone: one that
// holds a whole item writes its outputs, warps that share one leave partial results (running maximum, sum
// and weighted values in fp32), which a second kernel joins in the order of the tokens, so results do not
// depend on timing.
//
// Inside a warp:
//   - keys and values come into a ring of shared memory private to the warp (16-byte asynchronous copies,
//     kStages deep), tokens that no row sees as zeros;
//   - S^T = K Q^T and O^T += V^T P^T are fp16 tensor-core products of m16n8k16 fragments: tokens, then head
//     dimensions, fill the 16 rows, and the queries the 8 columns, so that few queries waste nothing.  (A
//     tcgen05 tile has 64 or 128 rows, and would need the codes widened in shared memory first.)  Each lane widens
//     exactly the codes of its own fragment in registers (e4m3 to fp16 is exact).  The order of the contraction index
//     is free, so a lane's 16 consecutive bytes of a key serve four k-steps, and its 16 consecutive dimensions of a
//     value eight row tiles: every shared-memory access is 16 bytes wide (8 for values at head_dim 64).  The weights
//     go from the scores' fragment layout to the operand's by 8 x 8 transposes (movmatrix);
//   - scales: a page's key exponent multiplies the scores; its value exponent e is folded into the weight,
//     w = 2^(s + e - m) with the reference m running over max(s + e), so that O accumulates w * code and
//     the sum takes w * 2^-e; nothing is lost whatever the pages' exponents.
//   - the reference m moves only when a weight would leave fp16 (see lift), so the rescale of O is rare.
//
// Measured (B200, copy rate 6.55 TB/s): 64 requests of 64 to 16384 tokens, 32/8 heads of 128: 79 us, 5.1 TB/s; 16 rows
// per key (verify, 4 drafts): 92 us for 363 MB, 3.9 TB/s.  At 8 rows per key a step is about 650 instructions
// issued at 44 % of the slots: latency is what is left.  Two blocks of rows need 240 registers, so eight warps an SM.
#include <math.h>

#include "attn_internal.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 32;                // tokens of a step
constexpr int kStages = 2;
constexpr int kItemSteps = 4;           // steps that beginning and ending an item takes the time of
// NB: blocks of 8 rows (of an item) that share each widened code: 1, 2 or 4.
// Blocks that an SM holds at a time, by registers and, for fp32's two parts of each query at D = 128, by shared memory
// (the kernel asserts the latter): the list is cut for exactly the warps that run at once.  fp32 at D = 128 cut for bf16's
// three blocks instead, of which two fit, had its last third wait for the rest: 64 requests of 64 to 16384 tokens, 32/8
// heads, 110 us against 84; 4 of 100001 to 131072, 32/4 heads, 131 against 97 (before fold_steps below: now 88 and 102).
constexpr int ctas_per_sm(int D, int NB, bool F32) {
    if (D == 128) return NB == 1 && !F32 ? 3 : 2;
    return NB == 1 ? 4 : NB == 2 ? 3 : 2;
}
constexpr int grid_size(int D, int NB, bool F32) { return kSMs * ctas_per_sm(D, NB, F32); }
constexpr int num_workers(int D, int NB, bool F32) { return grid_size(D, NB, F32) * kWarps; }

// Steps that the tensor core adds up at a time.  Its additions truncate, so that a long sum shrinks, by some 2^-25 of itself
// an addition (64 requests of 131072 tokens, 8 heads of 128: 1.4e-4 in fp32, of 1048576: 1.2e-3): what it holds is added to the
// warp's partial result in fp32 instructions every 512 tokens for fp32 (64 additions; 9e-7 for either) and every 4096 for
// bf16 (256; 6e-5).  Time: bf16 0 to 2 %, fp32 5 %.
template <bool F32> constexpr int fold_steps() { return F32 ? 16 : 128; }

constexpr int kJoinGrid = 4 * kSMs;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit values, two of row lane / 4 in each lane, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// copy16_or_zero at constant distances from two addresses, always live
template <int S, int G> __device__ __forceinline__ void copy16(uint32_t sdst, const uint8_t* gsrc) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(sdst), "l"(gsrc), "n"(S), "n"(G) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Position of 16-byte chunk `c` of token row `r` in a warp's tile.  The fragments read, in one access of 8
// lanes, chunks 0..3 of rows 2i and 2i+1 (keys), and one chunk pair of rows 0, 2, 4, 6 or 1, 3, 5, 7
// (values): the key makes both free of bank conflicts at head_dim 128.
template <int D> __device__ __forceinline__ uint32_t chunk_off(int r, int c) {
    if (D == 128) return r * 128 + ((c ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, int NB, bool F32> struct alignas(128) WarpSmem {
    static constexpr int kTile = kSub * D;  // bytes of one tile of keys or values
    uint8_t ring[kStages][2][kTile];
    uint32_t q[F32 ? 2 : 1][NB][D / 64][4][32][2];  // B fragments of the queries (high, low fp16 parts)
    float rs[8 * NB];                               // scale2 * 2^eq of each row
    float m_fold[8 * NB];                           // the reference of each row when its sums were last set aside
    int8_t exps[kStages][2][2];  // key and value exponents of a tile's two 16-token halves
    uint16_t anc[kMaxVerifyDraft];
    int8_t depth[kMaxVerifyDraft];
};

struct Request {
    int n, row0, L, kv, base;  // row0: first packed row; base: tokens before the new rows
    bool bad_len;              // a length outside the block table or below the row count
    bool dead;                 // that, or padding: its rows get zeros
    Range r;
    int nb;      // row blocks
    int a, b;    // visible tiles of 32 tokens: 0 .. a-1 and b ..
    int tiles;   // their count (1 for a dead request: its zeros)
    long long units;  // places in the list: kItemSteps and the tiles of each item
};

__device__ __forceinline__ Request get_request(const Args& p, int n, int rows_per_block) {
    Request q;
    q.n = n;
    if (p.cu) {
        q.row0 = p.cu[n];
        q.L = p.cu[n + 1] - q.row0;
    } else {
        q.row0 = n * p.per;
        q.L = p.per;
    }
    q.kv = p.kv_lens[n];
    q.bad_len = q.kv > 0 && (q.kv < q.L || (long long)q.kv > ((long long)p.max_pages << p.ps_shift));
    q.dead = q.kv <= 0 || q.bad_len;
    q.base = q.kv - q.L;
    q.nb = q.L * p.G <= p.rows_upto ? (q.L * p.G + rows_per_block - 1) / rows_per_block : 0;
    if (q.dead) {
        q.a = q.b = 0;
        q.tiles = 1;
        q.r = Range{0, 0, 0};
    } else {
        q.r = visible_range(p, n, q.kv, q.L);
        q.a = (q.r.pre + kSub - 1) / kSub;
        q.b = max(q.r.lo / kSub, q.a);
        q.tiles = q.a + (q.kv + kSub - 1) / kSub - q.b;
    }
    q.units = (long long)(q.tiles + kItemSteps) * q.nb * p.HKV;
    return q;
}

template <typename T, int D, int NB, Cap CAP>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NB, sizeof(T) == 4)) split_kernel(const __grid_constant__ Args p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int kRows = 8 * NB;
    constexpr int kDT = D / 16;  // row tiles of the output: dimensions
    constexpr int kFold = fold_steps<F32>();
    using S = WarpSmem<D, NB, F32>;
    constexpr int kParts = F32 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    // (beside the rings: s_sum below, and 1 KB that the system keeps)
    static_assert(ctas_per_sm(D, NB, F32) * (kWarps * sizeof(S) + 1152 + 1024) <= 228 * 1024,
                  "more blocks than an SM has shared memory for");
    const int lane = threadIdx.x & 31, worker = blockIdx.x * kWarps + (threadIdx.x >> 5), workers = gridDim.x * kWarps;
    S& sm = reinterpret_cast<S*>(smem_raw)[threadIdx.x >> 5];
    const int qr = lane >> 2, qc = lane & 3;  // fragment row (or column) and quad lane

    // ---- this warp's places [u0, u1) of all: every block scans the lengths for itself
    __shared__ long long s_sum[kThreads + 1];  // places before each thread's run of requests, and in all
    long long total, u0, u1, base, per;
    int n;
    {
        const int tid = threadIdx.x, chunk = (p.N + kThreads - 1) / kThreads;
        const int nb = tid * chunk, ne = min(p.N, nb + chunk);
        long long sum = 0;
        bool bad = p.cu && tid == 0 && p.cu[0] != 0;
#pragma unroll 4
        for (int i = nb; i < ne; ++i) {
            bool fits = true;
            if (p.cu) {
                const int c0 = p.cu[i], c1 = p.cu[i + 1];
                fits = c0 >= 0 && c1 >= c0 && c1 <= p.T;
            }
            bad = bad || !fits;
            if (fits) sum += get_request(p, i, kRows).units;
        }
        long long upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        s_sum[tid + 1] = upto;
        if (tid == 0) s_sum[0] = 0;
        bad = __syncthreads_or(bad) != 0;
        long long before = 0;  // of the warps before this one
        for (int w = 0; w < (tid >> 5); ++w) before += s_sum[32 * (w + 1)];
        __syncthreads();
        s_sum[tid + 1] = before + upto;
        __syncthreads();
        total = s_sum[kThreads];
        per = (total + workers - 1) / workers;
        u0 = per * worker;
        u1 = min(total, u0 + per);
        if (bad || u0 >= total) {
            if (lane == 0) {
                if (bad && worker == 0) raise_error(p.hdr, GDN_DEVERR_SEQLENS);
                p.meta[worker] = make_int4(-1, 0, 0, 0);
            }
            return;
        }
        int run = 0;  // the last run that begins at or before u0 and is not empty
        for (int i = lane; i < kThreads; i += 32)
            if (s_sum[i] <= u0 && u0 < s_sum[i + 1]) run = i;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) run = max(run, __shfl_xor_sync(0xffffffffu, run, o));
        base = s_sum[run];
        for (n = run * chunk;; ++n) {
            const long long units = get_request(p, n, kRows).units;
            if (u0 < base + units) break;
            base += units;
        }
    }
    let_next_launch_start();
    int4 meta = make_int4(-1, 0, 0, 0);
    const uint32_t ring_s = tc::smem_u32(sm.ring);
    const int ps_mask = (1 << p.ps_shift) - 1;

    long long u = u0;
    Request rq = get_request(p, n, kRows);
    while (u < u1) {
        if (u >= base + rq.units) {
            base += rq.units;
            rq = get_request(p, ++n, kRows);
            continue;
        }
        const int places = rq.tiles + kItemSteps;
        const int item = (int)((u - base) / places);
        const long long first_u = base + (long long)item * places + kItemSteps;  // the place of the item's first tile
        const int k0 = (int)max(0ll, u - first_u), k1 = (int)(min(u1, first_u + rq.tiles) - first_u);
        u = first_u + max(k1, 0);
        if (k1 <= 0) break;  // the piece ends before the item's first tile
        const int rb = item % rq.nb, h = item / rq.nb;
        const int rows = min(kRows, rq.L * p.G - rb * kRows);
        bool dead = rq.dead;

        // ---- the draft tree's ancestors (bit t': draft t' is t or an ancestor of t) and depths
        if (p.parents && !dead) {
            __syncwarp();
            bool ok = true;
            if (lane == 0)
                for (int t = 0; t < rq.L; ++t) {
                    const int par = p.parents[n * p.per + t];
                    if (par < -1 || par >= t) {
                        ok = false;
                        raise_error(p.hdr, GDN_DEVERR_TREE);
                        break;
                    }
                    sm.anc[t] = (uint16_t)((par < 0 ? 0 : sm.anc[par]) | (1u << t));
                    sm.depth[t] = (int8_t)(par < 0 ? 0 : sm.depth[par] + 1);
                }
            dead = !__all_sync(0xffffffffu, ok);
        }
        if (dead) {  // zeros, written by the warp that holds the item's first tile
            if (k0 == 0) {
                for (int e = lane; e < rows * D; e += 32) {
                    const int r = rb * kRows + e / D, t = p.token_of(r), hq = h * p.G + r - t * p.G;
                    static_cast<T*>(p.out)[((long long)(rq.row0 + t) * p.HQ + hq) * D + e % D] = from_f<T>(0.0f);
                }
                if (p.lse)
                    for (int e = lane; e < rows; e += 32) {
                        const int r = rb * kRows + e, t = p.token_of(r), hq = h * p.G + r - t * p.G;
                        p.lse[(long long)(rq.row0 + t) * p.HQ + hq] = -INFINITY;
                    }
                if (lane == 0 && rq.bad_len) raise_error(p.hdr, GDN_DEVERR_KV_LEN);
            }
            continue;
        }

        // ---- the ring.  Entry i is tile k0 + i; tile_tok gives its first token.
        const int steps = k1 - k0;
        auto tile_tok = [&](int i) {
            const int k = k0 + i;
            return (k < rq.a ? k : k - rq.a + rq.b) * kSub;
        };
        auto live = [&](int t) { return (t >= rq.r.lo && t < rq.kv) || t < rq.r.pre; };
        // page of token group [t, t + 16), -1 if no token of it is seen (aligned groups never span pages)
        auto page_of = [&](int t) -> int {
            if (!(t < rq.r.pre || (t < rq.kv && t + 15 >= rq.r.lo))) return -1;
            return __ldg(p.table + (long long)n * p.max_pages + (t >> p.ps_shift));
        };
        auto check_page = [&](int t, int pg) -> int {
            if (!(t < rq.r.pre || (t < rq.kv && t + 15 >= rq.r.lo))) return -1;
            if (pg >= 0 && pg < p.num_pages) return pg;
            if (lane == 0) raise_error(p.hdr, GDN_DEVERR_PAGE_RANGE);
            return -1;
        };
        int pg_next[2] = {-1, -1};  // pages of the entry that is fetched next (looked up one step ahead)
        int ex_val = 0, ex_entry = -1;  // lane 0..3: an exponent on its way to entry ex_entry
        constexpr int kPerRow = D / 16, kRowsEach = 32 / kPerRow;  // chunks of a row; rows of one copy instruction
        const int cr = lane / kPerRow, cc = lane % kPerRow;
        auto fetch = [&](int i) {
            if (i < steps) {
                const int t0 = tile_tok(i), st = i % kStages;
                const int pg0 = check_page(t0, pg_next[0]), pg1 = check_page(t0 + 16, pg_next[1]);
                const uint32_t dst = ring_s + st * (2 * S::kTile);
                if (pg0 >= 0 && pg1 >= 0 && ((t0 >= rq.r.lo && t0 + kSub <= rq.kv) || t0 + kSub <= rq.r.pre)) {
                    // all tokens are seen: two runs of 16 rows (a run lies within a page), constant distances inside
                    const long long o0 = ((((long long)pg0 * p.HKV + h) << p.ps_shift) + (t0 & ps_mask) + cr) * D + cc * 16;
                    const long long o1 = ((((long long)pg1 * p.HKV + h) << p.ps_shift) + ((t0 + 16) & ps_mask) + cr) * D + cc * 16;
                    // a lane's rows are kRowsEach apart: at D = 128 every other one lies on the other side of the swizzle's
                    // bit 2, at D = 64 all have the same place in the swizzle's period of 8
                    const uint32_t d0 = dst + chunk_off<D>(cr, cc), d1 = dst + chunk_off<D>(cr + kRowsEach, cc) - kRowsEach * D;
                    auto run = [&](uint32_t e, uint32_t f, const uint8_t* src) {
#define ATTN_COPY(J) copy16<(J) * kRowsEach * D, (J) * kRowsEach * D>((J) & 1 ? f : e, src)
                        ATTN_COPY(0);
                        ATTN_COPY(1);
                        if constexpr (kRowsEach == 4) {
                            ATTN_COPY(2);
                            ATTN_COPY(3);
                        }
#undef ATTN_COPY
                    };
                    run(d0, d1, p.k + o0);
                    run(d0 + 16 * D, d1 + 16 * D, p.k + o1);
                    run(d0 + S::kTile, d1 + S::kTile, p.v + o0);
                    run(d0 + S::kTile + 16 * D, d1 + S::kTile + 16 * D, p.v + o1);
                } else {
#pragma unroll 1
                    for (int j = 0; j < kSub / kRowsEach; ++j) {
                        const int r = j * kRowsEach + cr, pg = r < 16 ? pg0 : pg1, t = t0 + r;
                        const bool ok = pg >= 0 && live(t);
                        const long long off =
                            ok ? ((((long long)pg * p.HKV + h) << p.ps_shift) + (t & ps_mask)) * D + cc * 16 : 0;
                        copy16_or_zero(dst + chunk_off<D>(r, cc), p.k + off, ok);
                        copy16_or_zero(dst + S::kTile + chunk_off<D>(r, cc), p.v + off, ok);
                    }
                }
                const int pg = lane & 1 ? pg1 : pg0;
                const int8_t* e = lane & 2 ? p.v_exp : p.k_exp;
                ex_val = (lane < 4 && pg >= 0) ? (int)e[(long long)pg * p.HKV + h] : 0;
                ex_entry = i;
                if (i + 1 < steps) {
                    pg_next[0] = page_of(tile_tok(i + 1));
                    pg_next[1] = page_of(tile_tok(i + 1) + 16);
                }
            }
            copy_commit();
        };
        auto store_exp = [&]() {
            if (ex_entry >= 0 && lane < 4) sm.exps[ex_entry % kStages][lane >> 1][lane & 1] = (int8_t)ex_val;
            ex_entry = -1;
        };
        pg_next[0] = page_of(tile_tok(0));
        pg_next[1] = page_of(tile_tok(0) + 16);
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) {
            fetch(i);
            store_exp();
        }

        // ---- queries: 16 consecutive dimensions per lane, scaled by the row's power of two, into
        // fragment order (four k-steps of four dimensions each for lane (row % 8, chunk % 4))
        constexpr int kChunks = D / 16;
        #pragma unroll 4
        for (int r = lane / kChunks; r < kRows; r += 32 / kChunks) {
            const int c = lane % kChunks;
            const int rr = rb * kRows + r;
            float x[16];
            if (r < rows) {
                const int t = p.token_of(rr), hq = h * p.G + rr - t * p.G;
                const T* src = static_cast<const T*>(p.q) + (long long)(rq.row0 + t) * p.q_stride + hq * D + c * 16;
#pragma unroll
                for (int i = 0; i < 16; i += Vec16<T>::kN) Vec16<T>::get(*reinterpret_cast<const uint4*>(src + i), x + i);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 0.0f;
            }
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
            for (int o = 1; o < kChunks; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int eq = query_exponent(amax);
            if (c == 0) sm.rs[r] = p.scale2 * exp2i(eq);
            const float f = exp2i(-eq);
            const int fl = (r & 7) * 4 + (c & 3);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float y0 = x[4 * ks + 2 * i] * f, y1 = x[4 * ks + 2 * i + 1] * f;
                    const uint32_t hi = tc::pack_f16(y0, y1);
                    sm.q[0][r >> 3][c >> 2][ks][fl][i] = hi;
                    if constexpr (F32) {
                        const float2 b = tc::unpack_f16(hi);
                        sm.q[kParts - 1][r >> 3][c >> 2][ks][fl][i] = tc::pack_f16(y0 - b.x, y1 - b.y);
                    }
                }
        }
        __syncwarp();

        // ---- this lane's rows: fragment columns 2 qc and 2 qc + 1 of each block of 8
        constexpr int NR = 2 * NB;
        int pos[NR], anc[NR];
        float slope[NR], rs[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int own = 8 * (i >> 1) + 2 * qc + (i & 1), r = rb * kRows + own;
            const int t = min(p.token_of(r), rq.L - 1), hq = h * p.G + min(r - t * p.G, p.G - 1);
            rs[i] = sm.rs[own];
            slope[i] = p.slopes ? p.slopes[hq] * kLog2e : 0.0f;
            pos[i] = rq.base + (p.parents ? sm.depth[t] : t);
            anc[i] = p.parents ? sm.anc[t] : 0;
        }
        // every row sees the tokens up to seen_by_all (the window aside): in a tree, not even the first draft
        const int seen_by_all = p.parents ? rq.base - 1 : rq.base, pos_last = rq.base + rq.L - 1;
        const int window = p.window > 0 ? p.window : 0x7fffffff, prefix = p.prefix ? p.prefix[n] : 0;
        const bool modified = p.cap2 > 0.0f || p.slopes;  // scores are more than scaled
        const float cap_in = 2.0f * kLog2e / p.cap2;

        float m[NR], l[NR], o[NB][kDT][4];
#pragma unroll
        for (int i = 0; i < NR; ++i) m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int d = 0; d < kDT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][d][e] = 0.0f;

        // Adds the lane's sums, dim(d) and the seven dimensions behind it for d = 0, 4, .., to what has been set aside of the item, if
        // anything: there (keep) or in the registers.
        auto slot_of = [&] { return (long long)(worker * 2 + (k0 == 0 ? 1 : 0)) * kRows; };
        auto fold = [&](bool any, bool keep) {
            int first = (int)slot_of() + 2 * qc;
            asm volatile("" : "+r"(first));  // formed here, not kept in registers through the steps
            float* const mine = p.part_o + (long long)first * D + qr * (D / 8);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = 8 * (i >> 1) + 2 * qc + (i & 1);
                const float mf = any ? sm.m_fold[r] : 0.0f, f = mf == -INFINITY ? 0.0f : tc::ex2_approx(mf - m[i]);
                float4* at = reinterpret_cast<float4*>(mine + (8 * (i >> 1) + (i & 1)) * D);  // 4 dimensions each
                float4 y[kDT / 2];
#pragma unroll
                for (int d = 0; d < kDT / 2; ++d) y[d] = any ? at[d] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int d = 0; d < kDT / 2; ++d) {
                    float& x0 = o[i >> 1][2 * d][i & 1];
                    float& x1 = o[i >> 1][2 * d][2 + (i & 1)];
                    float& x2 = o[i >> 1][2 * d + 1][i & 1];
                    float& x3 = o[i >> 1][2 * d + 1][2 + (i & 1)];
                    x0 = fmaf(y[d].x, f, x0), x1 = fmaf(y[d].y, f, x1), x2 = fmaf(y[d].z, f, x2), x3 = fmaf(y[d].w, f, x3);
                    if (keep) {
                        at[d] = make_float4(x0, x1, x2, x3);
                        x0 = x1 = x2 = x3 = 0.0f;
                    }
                }
            }
            __syncwarp();
            if (keep && qr == 0)
#pragma unroll
                for (int i = 0; i < NR; ++i) sm.m_fold[8 * (i >> 1) + 2 * qc + (i & 1)] = m[i];
        };

        int it = 0;
        do {  // a loop of its own for what the tensor core adds up: the rare rest costs the steps no registers
            do {
                copy_wait<kStages - 2>();
                store_exp();
                __syncwarp();  // the entry has landed for every lane, and the one before it has been read by all
                fetch(it + kStages - 1);

                const int st = it % kStages, t0 = tile_tok(it);
                const uint8_t* ks = sm.ring[st][0];
                const uint8_t* vs = sm.ring[st][1];
                const float kf[2] = {exp2i(sm.exps[st][0][0]), exp2i(sm.exps[st][0][1])};
                const int ve[2] = {sm.exps[st][1][0], sm.exps[st][1][1]};

                // S^T[16 tokens][block of rows]: element e is token 16 j + 8 (e / 2) + qr, row 2 qc + e % 2
                float s[2][NB][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[j][nb][e] = 0.0f;
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh) {
                    uint32_t kw[4][4];  // rows 8 j + qr
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 w = *reinterpret_cast<const uint4*>(ks + chunk_off<D>(8 * j + qr, qc + 4 * hh));
                        kw[j][0] = w.x, kw[j][1] = w.y, kw[j][2] = w.z, kw[j][3] = w.w;
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        uint2 b[kParts][NB];
#pragma unroll
                        for (int part = 0; part < kParts; ++part)
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                b[part][nb] = *reinterpret_cast<const uint2*>(sm.q[part][nb][hh][kk][lane]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w0 = kw[2 * j][kk], w1 = kw[2 * j + 1][kk];
                            const uint32_t a[4] = {widen_lo(w0), widen_lo(w1), widen_hi(w0), widen_hi(w1)};
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) mma16816(s[j][nb], a, b[part][nb].x, b[part][nb].y);
                        }
                    }
                }

                // scores in base-2 units plus the value exponent
                const bool whole = (t0 + kSub - 1 <= seen_by_all && pos_last - t0 < window) || t0 + kSub <= rq.r.pre;
                if (whole && !p.slopes) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < NR; ++i) {
                            const float a = fminf(rs[i] * kf[j], 3.0e38f);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float& x = s[j][i >> 1][2 * e + (i & 1)];
                                if (p.cap2 > 0.0f) x = capped<CAP>(x * a, p.cap2, cap_in) + (float)ve[j];
                                else x = fmaf(x, a, (float)ve[j]);
                            }
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = t0 + 16 * j + 8 * e + qr;
                            int at = t, draft = -1;  // the token's position, and which draft of a tree it is
                            if (p.parents && t >= rq.base) {
                                draft = min(t - rq.base, rq.L - 1);
                                at = rq.base + sm.depth[draft];
                            }
                            const bool always = t < prefix;
#pragma unroll
                            for (int i = 0; i < NR; ++i) {
                                float& x = s[j][i >> 1][2 * e + (i & 1)];
                                const float a = fminf(rs[i] * kf[j], 3.0e38f);
                                if (modified) {
                                    x *= a;
                                    if (p.cap2 > 0.0f) x = capped<CAP>(x, p.cap2, cap_in);
                                    x = fmaf(-slope[i], fabsf((float)(pos[i] - at)), x) + (float)ve[j];
                                } else {
                                    x = fmaf(x, a, (float)ve[j]);  // as above: a mask changes no bit of what is seen
                                }
                                bool sees = draft >= 0 ? (anc[i] >> draft) & 1 : t <= pos[i];
                                sees = ((sees && pos[i] - at < window) || always) && t < rq.kv;
                                x = sees ? x : -INFINITY;
                            }
                        }
                }
                float mx[NR];
                bool move = false;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    mx[i] = max3(fmaxf(s[0][i >> 1][i & 1], s[0][i >> 1][2 + (i & 1)]), s[1][i >> 1][i & 1], s[1][i >> 1][2 + (i & 1)]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
                    move = move || mx[i] > m[i] + kMaxWeight;
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        if (mx[i] > m[i] + kMaxWeight) {
                            const float f = tc::ex2_approx(m[i] - (mx[i] - lift<F32>()));  // 0 from m = -inf
                            m[i] = mx[i] - lift<F32>();
                            l[i] *= f;
#pragma unroll
                            for (int d = 0; d < kDT; ++d) {
                                o[i >> 1][d][i & 1] *= f;
                                o[i >> 1][d][2 + (i & 1)] *= f;
                            }
                        }
                    }
                }
                // weights; a row that has seen nothing keeps m = -inf and takes 0 as its reference
                const float vf[2] = {exp2i(-ve[0]), exp2i(-ve[1])};
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float ref = m[i] == -INFINITY ? 0.0f : m[i];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& x0 = s[j][i >> 1][i & 1];
                        float& x1 = s[j][i >> 1][2 + (i & 1)];
                        x0 = tc::ex2_approx(x0 - ref);
                        x1 = tc::ex2_approx(x1 - ref);
                        l[i] = fmaf(x0 + x1, vf[j], l[i]);
                    }
                }

                // O^T += V^T P^T, 16 tokens at a time
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t b[kParts][NB][2];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x0 = s[j][nb][2 * e], x1 = s[j][nb][2 * e + 1];
                            const uint32_t w = tc::pack_f16(x0, x1);
                            b[0][nb][e] = transpose8x8(w);
                            if constexpr (F32) {
                                const float2 r = tc::unpack_f16(w);
                                b[kParts - 1][nb][e] = transpose8x8(tc::pack_f16(x0 - r.x, x1 - r.y));
                            }
                        }
                    constexpr int kW = D / 32;  // words of a lane's D/8 dimensions of one token
                    uint32_t w[4][kW];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * j + 2 * qc + (i & 1) + 8 * (i >> 1);
                        if constexpr (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(vs + chunk_off<D>(r, qr));
                            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(vs + chunk_off<D>(r, qr >> 1) + (qr & 1) * 8);
                            w[i][0] = x.x, w[i][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < kW; ++x)
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            // bytes 2 d and 2 d + 1 of two tokens interleaved: dimensions 4 x + 2 d and the next are the row
                            // tile's rows qr and qr + 8
                            const uint32_t lo = __byte_perm(w[0][x], w[1][x], d ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(w[2][x], w[3][x], d ? 0x7362 : 0x5140);
                            const uint32_t a[4] = {widen_lo(lo), widen_hi(lo), widen_lo(hi), widen_hi(hi)};
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][2 * x + d], a, b[part][nb][0], b[part][nb][1]);
                        }
                }
            } while (++it < steps && it % kFold != 0);
            if (steps > kFold) fold(it > kFold, it < steps);
        } while (it < steps);
        copy_wait<0>();

        // ---- results: a lane holds D/8 consecutive dimensions of each of its rows
        const bool complete = k0 == 0 && k1 == rq.tiles;
        const long long slot = slot_of();
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
            const int r = 8 * (i >> 1) + 2 * qc + (i & 1);
            if (r >= rows) continue;
            const int rr = rb * kRows + r, t = p.token_of(rr), hq = h * p.G + rr - t * p.G;
            const long long row = (long long)(rq.row0 + t) * p.HQ + hq;
            const float f = !complete ? 1.0f : l[i] == 0.0f ? 0.0f : 1.0f / l[i];
            if (qr == 0) {
                if (!complete) p.part_ml[slot + r] = make_float2(m[i], l[i]);
                else if (p.lse) p.lse[row] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
            }
#pragma unroll
            for (int d = 0; d < kDT; d += 4) {
                float y[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) y[x] = o[i >> 1][d + (x >> 1)][2 * (x & 1) + (i & 1)] * f;
                const int dim = qr * (D / 8) + 2 * d;
                if (complete) {
                    T* at = static_cast<T*>(p.out) + row * D + dim;
#pragma unroll
                    for (int x = 0; x < 8; x += Vec16<T>::kN) *reinterpret_cast<uint4*>(at + x) = Vec16<T>::put(y + x);
                } else {
                    float* at = p.part_o + (slot + r) * D + dim;
                    *reinterpret_cast<float4*>(at) = make_float4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<float4*>(at + 4) = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
        }
        if (!complete && k0 == 0) meta = make_int4(n, h, rb, (int)((first_u + rq.tiles - 1) / per));
        __syncwarp();  // shared memory is reused by the next item
    }
    if (lane == 0) p.meta[worker] = meta;
}

// Joins the partial results of the items that begin in a warp and go on in others, in the order of the warps: block
// (i, r) handles row r of those of warps i, i + gridDim.x, ...
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args p, int rows_per_block, int workers) {
    __shared__ float wts[num_workers(64, 1, false)];  // the most of all forms
    __shared__ float red[8];
    __shared__ float acc[128 * 4];
    const int tid = threadIdx.x, r = blockIdx.y;
    wait_for_launch_before();
    for (int first = blockIdx.x; first < workers; first += gridDim.x) {
        const int4 meta = p.meta[first];
        if (meta.x < 0) continue;
        const int h = meta.y, count = meta.w - first + 1;
        const int L = p.cu ? p.cu[meta.x + 1] - p.cu[meta.x] : p.per, row0 = p.cu ? p.cu[meta.x] : meta.x * p.per;
        const int rr = meta.z * rows_per_block + r;
        if (rr >= L * p.G) continue;
        auto slot = [&](int i) { return (long long)((first + i) * 2 + (i == 0 ? 1 : 0)) * rows_per_block + r; };
        float mm = -INFINITY;
        for (int i = tid; i < count; i += 128) mm = fmaxf(mm, p.part_ml[slot(i)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        if ((tid & 31) == 0) red[tid >> 5] = mm;
        __syncthreads();
        mm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        float ll = 0.0f;
        for (int i = tid; i < count; i += 128) {
            const float2 x = p.part_ml[slot(i)];
            const float f = x.x == -INFINITY ? 0.0f : tc::ex2_approx(x.x - mm);
            wts[i] = f;
            ll += x.x == -INFINITY ? x.y : x.y * f;
        }
        ll = warp_sum(ll);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = ll;
        __syncthreads();
        ll = red[4] + red[5] + red[6] + red[7];
        constexpr int kCols = D / 4, kGroups = 128 / kCols;
        const int c = tid % kCols, g = tid / kCols;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = g; i < count; i += kGroups) {
            const float4 y = reinterpret_cast<const float4*>(p.part_o + slot(i) * D)[c];
            const float f = wts[i];
            x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
        }
        reinterpret_cast<float4*>(acc)[tid] = x;
        __syncthreads();
        if (tid < D) {
            float y = 0.0f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) y += acc[i * D + tid];
            const int t = p.token_of(rr), hq = h * p.G + rr - t * p.G;
            const long long row = (long long)(row0 + t) * p.HQ + hq;
            static_cast<T*>(p.out)[row * D + tid] = from_f<T>(ll == 0.0f ? 0.0f : y / ll);
            if (p.lse && tid == 0) p.lse[row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        }
        __syncthreads();
    }
}

template <typename T, int D, int NB, Cap CAP>
cudaError_t launch_cap(const Args& p, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    static_assert(num_workers(D, NB, F32) <= num_workers(64, 1, false), "the join holds a weight for each warp");
    const int smem = kWarps * (int)sizeof(WarpSmem<D, NB, F32>);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(split_kernel<T, D, NB, CAP>), smem, done);
    if (e != cudaSuccess) return e;
    split_kernel<T, D, NB, CAP><<<grid_size(D, NB, F32), kThreads, smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(join_kernel<T, D>, dim3(kJoinGrid, 8 * NB), 128, 0, s, p, 8 * NB, num_workers(D, NB, F32));
}

// CAP is the form of a cap if there is one: whether there is, the kernel asks for itself
template <typename T, int D, int NB>
cudaError_t launch_rows(const Args& p, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    if constexpr (!F32)
        if (cap_form<F32>(p.cap2) != kTanhCap) return launch_cap<T, D, NB, kExpCap>(p, s);
    return launch_cap<T, D, NB, kTanhCap>(p, s);
}

template <typename T, int D>
cudaError_t launch_dim(const Args& p, cudaStream_t s) {
    // rows that read each key, in blocks of 8: one, two or four share each widened code
    const long long rows = p.cu ? (long long)p.T * p.G / (p.N > 0 ? p.N : 1) : (long long)p.per * p.G;
    if constexpr (split_rows(D, sizeof(T) == 4) > 16)
        if (rows > 16) return launch_rows<T, D, 4>(p, s);
    return rows > 8 ? launch_rows<T, D, 2>(p, s) : launch_rows<T, D, 1>(p, s);
}

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

// partial results: two for each warp, of the rows of a block
struct Layout {
    size_t meta, part_o, part_ml;
    explicit Layout(int D) {
        size_t warps = 0, rows = 0;
        for (int nr = 1; nr <= 4; nr *= 2) {
            const size_t w = (size_t)num_workers(D, nr, false);  // bf16 has as many warps as fp32 or more
            warps = w > warps ? w : warps;
            rows = w * 8 * nr > rows ? w * 8 * nr : rows;
        }
        meta = round16(warps * sizeof(int4));
        part_o = 2 * rows * (size_t)D * sizeof(float);
        part_ml = 2 * rows * sizeof(float2);
    }
};

}  // namespace

size_t split_workspace_bytes(int D) {
    const Layout y(D);
    return kHeaderBytes + y.meta + y.part_o + y.part_ml;
}

cudaError_t launch_split(Args p, int D, int dtype, cudaStream_t s) {
    const Layout y(D);
    uint8_t* w = reinterpret_cast<uint8_t*>(p.hdr) + kHeaderBytes;
    p.meta = reinterpret_cast<int4*>(w);
    p.part_o = reinterpret_cast<float*>(w + y.meta);
    p.part_ml = reinterpret_cast<float2*>(w + y.meta + y.part_o);
    if (dtype == GDN_DTYPE_F32) return D == 128 ? launch_dim<float, 128>(p, s) : launch_dim<float, 64>(p, s);
    return D == 128 ? launch_dim<__nv_bfloat16, 128>(p, s) : launch_dim<__nv_bfloat16, 64>(p, s);
}

}  // namespace attn
}  // namespace gdn
