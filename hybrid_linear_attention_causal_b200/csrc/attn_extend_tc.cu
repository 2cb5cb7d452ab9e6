// Attention of many new rows over the 8-bit paged cache (extend), on the tcgen05 tensor cores.
//
// An item is 256 rows of one key/value head of one request (rows are (new row, query head of the group)
// pairs, so that every row of an item reads the same keys; 128 rows for fp32), against its visible tokens in
// tiles of 128.  All (item, tile) units form one list that is cut into equal pieces, one per CTA of a
// persistent grid; a planning kernel lays the list out from the device's lengths.  An item that two or more
// CTAs share leaves partial results, joined afterwards in token order.
//
// Roles inside a CTA:
//   warps 0-3, 4-7  softmax of the item's rows 0-127 and 128-255 ("streams" 0 and 1), a row per thread
//   warps 8-11      widen the codes to fp16 and store them as swizzled operand tiles
//   warp 15         issues the products: S = Q K^T into tensor memory (SS), O += P V (A = P from tensor memory)
//   warp 12         copies the tile's codes into shared memory (bulk copies of 16 tokens) and its exponents
//   warp 14         copies the queries to where the streams convert them
//   warp 13         lays out the segments (items or parts of them) of this CTA ahead of their use
// While one stream's softmax runs, the tensor core works for the other: 2 x 2 x 128 x 128 x D products per
// tile against 2 x 128 x 128 exponentials, which at 16 a clock and SM take as long as the products at D = 128.
// Scores are kept in base-2 units; scales, the running reference and the weights are those of attn_split.cu.
// For fp32 the queries and the weights are two fp16 each (one stream, two products for each one), and O is added up in
// fp32 instructions every 4 tiles (in the idle stream's columns): the tensor core's own additions
// truncate, which over hundreds of tiles would cost more than fp32's rounding (3e-6 over 5000 tokens).  bf16 does so every
// 256 tiles, through global memory: behind a million tokens its outputs had shrunk by 0.29 %, more than their rounding (now
// 0.01 %; 2 % of the time of such calls, and of capped ones, is what the code for it takes).
//
// An item with at most 128 rows (the end of a sequence, a verify pass) has both streams work on the same rows, one
// on the even and one on the odd tiles ("twin"); stream 0 joins the two results in the end: rows r of both lie in the
// same lanes of tensor memory (through global memory instead, and with the trees' ancestors read by every row's thread,
// 64 requests of 64 rows over 375021 tokens took 128 us in place of 110).
//
// Measured (B200, 1633 TFLOP/s): 8192 rows behind 8192 tokens, 16/2 heads of 128: 810 to 860 us, 0.96 to 1.02 PFLOP/s; 18114
// rows in 8 sequences, 32/8 heads: 670 to 690 us, 0.65 to 0.67 PFLOP/s.  A unit of 256 rows and 128 tokens takes 3850 clocks against 2048 of
// products: each stream alternates between its softmax (2100) and its products, and the two overlap.  The loops'
// code has to stay small: unrolled further (171 KB), instruction fetches alone cost a third, and four times
// unrolled widening and eight times unrolled copies of queries still cost 7 % of the second case (728 us).
//
// Shared memory at D = 128: 64 KB of queries, two stages of keys and of values at 32 KB each, 32 KB of codes: one CTA per SM.
// Tensor memory: S of both streams (128 columns each; P takes the place of S), O of both (D columns each).
#include <math.h>

#include "attn_internal.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {
namespace {

constexpr int kTile = 128;   // tokens of a tile
constexpr int kThreads = 16 * 32;
// registers a thread: 512 x 128 at launch, shared out anew between the softmax and the other warps
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs <= 4 * 128, "more registers than the block is launched with");
// Tiles whose values the tensor core adds up at a time (8 additions each, 16 for fp32): its additions truncate (see
// attn_split.cu).  bf16: at 64 tiles the sums set aside cost extend_long's items of 64 to 128 tiles 5 %.
template <bool F32> constexpr int fold_tiles() { return F32 ? 4 : 256; }
constexpr int kExpSlots = 4; // tiles whose exponents are held
constexpr int kGrid = kSMs;

template <bool F32> constexpr int item_rows() { return F32 ? 128 : 256; }

struct Geometry {  // a request
    int row0, L, kv, base;
    bool bad_len, dead;
};

__device__ __forceinline__ Geometry geometry(const Args& p, int n) {
    Geometry g;
    g.row0 = p.cu ? p.cu[n] : n * p.per;
    g.L = p.cu ? p.cu[n + 1] - g.row0 : p.per;
    g.kv = p.kv_lens[n];
    g.base = g.kv - g.L;
    g.bad_len = g.kv > 0 && (g.kv < g.L || (long long)g.kv > ((long long)p.max_pages << p.ps_shift));
    g.dead = g.kv <= 0 || g.bad_len;  // (a bad tree is found when its segments are laid out)
    return g;
}

// The tiles that rows [r0, r0 + count) of a request see: 0 .. a-1 and b .. ; `tiles` of them.
struct Tiles {
    int lo, pre, a, b, tiles;
};

__device__ __forceinline__ Tiles tiles_of(const Args& p, int n, const Geometry& g, int r0, int count) {
    Tiles t;
    // a draft of a tree may stand anywhere from the first draft's position on
    const int first = g.base + (p.parents ? 0 : p.token_of(r0)), last = g.base + p.token_of(r0 + count - 1);
    t.pre = p.prefix ? max(0, min(p.prefix[n], g.kv)) : 0;
    t.lo = p.window > 0 ? max(0, first + 1 - p.window) : 0;
    const int hi = max(last + 1, t.pre);
    if (t.pre >= t.lo) t.lo = 0;
    t.a = t.lo > 0 ? (t.pre + kTile - 1) / kTile : 0;
    t.b = max(t.lo / kTile, t.a);
    t.tiles = t.a + (hi + kTile - 1) / kTile - t.b;
    return t;
}

// ---- the list of units: items[i] = (request, row tile), prefix[i] = units of one head before item i
__global__ void __launch_bounds__(1024) plan_kernel(const __grid_constant__ Args p, int item_rows) {
    let_next_launch_start();
    __shared__ long long s_warp[32];
    __shared__ long long s_carry;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // exclusive scan over the block of one value per thread, added to the running carry
    auto scan = [&](long long x) -> long long {
        long long inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            long long w = s_warp[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += y;
            }
            s_warp[lane] = w;
        }
        __syncthreads();
        const long long before = s_carry + (warp ? s_warp[warp - 1] : 0) + inc - x;
        const long long all = s_warp[31];
        __syncthreads();
        if (tid == 0) s_carry += all;
        __syncthreads();
        return before;
    };
    if (tid == 0) s_carry = 0;
    bool bad = p.cu && tid == 0 && p.cu[0] != 0;
    if (p.cu)
        for (int n = tid; n < p.N; n += 1024) {
            const int c0 = p.cu[n], c1 = p.cu[n + 1];
            bad = bad || c0 < 0 || c1 < c0 || c1 > p.T;
        }
    bad = __syncthreads_or(bad) != 0;
    if (bad) {
        if (tid == 0) {
            raise_error(p.hdr, GDN_DEVERR_SEQLENS);
            p.plan[0] = 0;
        }
        return;
    }
    for (int n0 = 0; n0 < p.N; n0 += 1024) {
        const int n = n0 + tid;
        int nb = 0;
        if (n < p.N) {
            const int rows = (p.cu ? p.cu[n + 1] - p.cu[n] : p.per) * p.G;
            nb = rows > p.rows_above ? (rows + item_rows - 1) / item_rows : 0;
        }
        const long long at = scan(nb);
        if (n < p.N) {
            for (int i = 0; i < nb; ++i) p.items[at + i] = make_int2(n, i);
        }
    }
    const int count = (int)s_carry;
    __syncthreads();
    if (tid == 0) s_carry = 0;
    __syncthreads();
    for (int i0 = 0; i0 < count; i0 += 1024) {
        const int i = i0 + tid;
        int units = 0;
        if (i < count) {
            const int2 it = p.items[i];
            const Geometry g = geometry(p, it.x);
            units = g.dead ? 1
                           : tiles_of(p, it.x, g, it.y * item_rows, min(item_rows, g.L * p.G - it.y * item_rows)).tiles;
        }
        const long long at = scan(units);
        if (i < count) p.prefix_units[i] = at;
    }
    if (tid == 0) {
        p.prefix_units[count] = s_carry;
        p.plan[0] = count;
    }
}

struct Segment {
    Geometry g;
    Tiles t;
    int n, h, rb, rows;
    int k0, k1;      // its tiles, of t.tiles
    int steps;       // k1 - k0, 0 for a dead request
    int nt[2];       // tiles of each stream: the first ones, or every other one (twin)
    bool twin;       // both streams have the same rows
    bool first, last;
    bool bad_tree;   // (then dead too)
    int end_cta;     // the CTA that holds the item's last unit
};

struct Tree {  // of each draft: its ancestors and itself, and its depth
    uint16_t anc[kMaxVerifyDraft];
    int8_t depth[kMaxVerifyDraft];
};

// Walks the segments (items or parts of them) of one CTA's piece of the list, a whole warp at once.
template <int kRows, bool kTwin> struct Walk {
    long long u, u1, per, head_units;
    int item, count, h;
    uint32_t anc = 0;  // of a tree: bit t is set where draft t is draft `lane` or an ancestor of it
    __device__ __forceinline__ bool begin(const Args& p) {
        const int lane = threadIdx.x & 31;
        count = p.plan[0];
        if (count == 0) return false;
        head_units = p.prefix_units[count];
        const long long total = head_units * p.HKV;
        per = (total + gridDim.x - 1) / gridDim.x;
        u = per * blockIdx.x;
        u1 = min(total, u + per);
        if (u >= u1) return false;
        h = (int)(u / head_units);
        const long long r = u - h * head_units;
        int lo = 0, n = count;  // the last item with prefix <= r (every item has a unit) is one of lo .. lo + n - 1:
        while (n > 1) {         // a load for every 32nd part of them, since each round waits for memory once
            const int part = (n + 31) >> 5, at = lane * part;
            const int upto = __popc(__ballot_sync(0xffffffffu, at < n && p.prefix_units[lo + at] <= r)) - 1;
            lo += upto * part;
            n = min(part, n - upto * part);
        }
        item = lo;
        return true;
    }
    __device__ __forceinline__ bool next(const Args& p, Segment& s) {
        if (u >= u1) return false;
        if (item == count) {
            item = 0;
            ++h;
        }
        const int2 it = p.items[item];
        const long long start = p.prefix_units[item] + h * head_units, end = p.prefix_units[item + 1] + h * head_units;
        s.n = it.x;
        s.rb = it.y;
        s.h = h;
        s.g = geometry(p, s.n);
        s.bad_tree = false;
        if (p.parents && !s.g.dead) {
            const int lane = threadIdx.x & 31;
            int up = lane < s.g.L ? p.parents[s.n * p.per + lane] : -1;
            s.bad_tree = s.g.dead = __any_sync(0xffffffffu, up < -1 || up >= lane);
            anc = 1u << lane;
#pragma unroll
            for (int i = 1; i < kMaxVerifyDraft; i <<= 1) {  // after a round twice as many generations
                const uint32_t a = __shfl_sync(0xffffffffu, anc, max(up, 0));
                const int next = __shfl_sync(0xffffffffu, up, max(up, 0));
                if (up >= 0) anc |= a, up = next;
            }
        }
        s.rows = min(kRows, s.g.L * p.G - s.rb * kRows);
        s.k0 = (int)(u - start);
        s.k1 = (int)(min(end, u1) - start);
        s.first = s.k0 == 0;
        s.last = start + s.k1 == end;
        s.end_cta = (int)((end - 1) / per);
        s.nt[0] = s.nt[1] = s.steps = 0;
        s.twin = kTwin && s.rows <= 128;
        if (!s.g.dead) {
            s.t = tiles_of(p, s.n, s.g, s.rb * kRows, s.rows);
            s.nt[0] = s.steps = s.k1 - s.k0;
            if (s.twin) {
                s.nt[0] = (s.steps + 1) >> 1;
                s.nt[1] = s.steps >> 1;
            } else if (s.rows > 128) {
                // stream 0's rows come first: the tiles behind its last visible token are stream 1's alone
                s.nt[1] = s.steps;
                const int hi0 = max(s.g.base + p.token_of(s.rb * kRows + 127) + 1, s.t.pre);
                const int end0 = (hi0 + kTile - 1) / kTile - s.t.b + s.t.a;
                s.nt[0] = max(0, min(s.k1, end0) - s.k0);
            }
        }
        u = start + s.k1;
        ++item;
        return true;
    }
};

constexpr int kSegSlots = 4;  // segments laid out ahead

template <int D, int kRows> struct Smem {
    uint8_t q[2][128 * D * 2];  // streams 0 and 1 (fp32: high and low parts)
    uint8_t k[2][kTile * D * 2];
    uint8_t v[2][kTile * D * 2];
    uint8_t raw[2][kTile * D];  // codes of the next tile's keys and values
    float4 scale[kExpSlots][kTile / 16];  // of each 16 tokens: 2^(key exponent), value exponent, 2^-(value exponent)
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], qfull[2], qraw[2], qempty[2], sfull[2], pfull[2], ofull[2], rfull[2], rempty[2], tfull, tempty, drained;
    uint64_t segfull[kSegSlots], segempty[kSegSlots];
    uint32_t tmem;
    Segment seg[kSegSlots];
    Tree tree[kSegSlots];
    int more[kSegSlots];  // 0: the list has ended
    float2 twin_ml[128];   // stream 1's maxima and sums, for stream 0
};

// 16 codes as 16 fp16
__device__ __forceinline__ void widen16(uint4 c, uint4& lo, uint4& hi) {
    lo = make_uint4(widen_lo(c.x), widen_hi(c.x), widen_lo(c.y), widen_hi(c.y));
    hi = make_uint4(widen_lo(c.z), widen_hi(c.z), widen_lo(c.w), widen_hi(c.w));
}
// Where 8 consecutive dimensions (chunk c) stand in a tile's row: the second 64 dimensions with neighbouring chunks
// exchanged, so that the even chunks of both halves, written together, lie in different banks.
__device__ __forceinline__ constexpr int chunk_of(int c) { return c ^ ((c >> 3) & 1); }

template <int R> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// 32 lanes x 32 columns of tensor memory, without the wait
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// two fp32 at a time
__device__ __forceinline__ void fma2(float& x0, float& x1, float a, float b) {  // x = x * a + b
    asm("{\n\t.reg .b64 x, a, b;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, a, b;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
    asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 s, s, x;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "f"(x0), "f"(x1));
}

// 16 scores scaled and capped.  (A polynomial tanh for scores below the cap, in place of two more visits to the unit
// of the exponentials, was no faster.)
template <Cap CAP> __device__ __forceinline__ void cap16(float* x, float a, float cap2, float cap_in) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = capped<CAP>(x[i] * a, cap2, cap_in);
}

template <typename T, int D, Cap CAP>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const __grid_constant__ Args p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int kRows = item_rows<F32>();
    constexpr int kSteps = D / 16;  // k-steps of Q K^T
    constexpr int kFold = fold_tiles<F32>();
    constexpr uint32_t kIdS = tc::idesc_f16(128, kTile), kIdO = tc::idesc_f16(128, D) | tc::kTransposeB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, kRows>& sm = *reinterpret_cast<Smem<D, kRows>*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 0) tc::tmem_alloc(&sm.tmem, 512);
    if (tid == 32) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&sm.kfull[i]), 4);
            tc::mbar_init(tc::smem_u32(&sm.vfull[i]), 4);
            tc::mbar_init(tc::smem_u32(&sm.kempty[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.vempty[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.qfull[i]), 4);
            tc::mbar_init(tc::smem_u32(&sm.qraw[i]), 32);
            tc::mbar_init(tc::smem_u32(&sm.qempty[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.sfull[i]), 2);
            tc::mbar_init(tc::smem_u32(&sm.pfull[i]), 4);
            tc::mbar_init(tc::smem_u32(&sm.ofull[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.rfull[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.rempty[i]), 4);
        }
        tc::mbar_init(tc::smem_u32(&sm.drained), 1);
        tc::mbar_init(tc::smem_u32(&sm.tfull), 4);
        tc::mbar_init(tc::smem_u32(&sm.tempty), 4);
        for (int i = 0; i < kSegSlots; ++i) {
            tc::mbar_init(tc::smem_u32(&sm.segfull[i]), 1);
            tc::mbar_init(tc::smem_u32(&sm.segempty[i]), 15);  // softmax 8, products 1, widening 4, copies 1, queries 1
        }
        tc::fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // an allocation of all 512 columns starts at column 0 (known to the compiler, the address costs the issuer nothing)
    constexpr uint32_t tm = 0;
    bool ok = sm.tmem == tm;
    int4 meta = make_int4(-1, 0, 0, 0);
    wait_for_launch_before();  // the plan
    let_next_launch_start();
    // the next segment, laid out by warp 13 (null: the list has ended), and its return
    uint32_t n_seg = 0;
    auto take = [&]() -> const Segment* {
        ok = ok && tc::mbar_wait(tc::smem_u32(&sm.segfull[n_seg % kSegSlots]), (n_seg / kSegSlots) & 1);
        const uint32_t at = n_seg++ % kSegSlots;
        return ok && sm.more[at] ? &sm.seg[at] : nullptr;
    };
    auto give = [&](const Segment* q) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.segempty[q - sm.seg]));
    };
    uint32_t tile = 0;  // tiles of the segments before this one: the stages' and slots' counter

    if (warp < 8) regs_up<kSoftmaxRegs>();
    else regs_down<kOtherRegs>();
    if (warp < 8) {
        // ---------------- softmax: thread = row
        const int st = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t tS = tm + lanes + st * 128, tO = tm + lanes + 256 + st * 128;
        const uint32_t tP = F32 ? tm + lanes + 128 : tS, tSum = tm + lanes + 384;
        uint32_t n_s = 0, n_o = 0, n_q = 0, n_t = 0;
        bool owed = false;  // stream 1: stream 0 has yet to read this one's accumulator (twin)
        // Queries of a segment: the rows that warp 14 has brought, each scaled by its power of two and rounded to fp16 in
        // place by its thread (fp32: 4 dimensions of either tile make 8 high and 8 low parts).  Where a row's chunks
        // stand does not matter here.  Returns the row's scale.
        auto queries = [&](const Segment& s) -> float {
            ok = ok && tc::mbar_wait(tc::smem_u32(&sm.qraw[st]), n_q++ & 1);
            uint8_t *q0 = sm.q[F32 ? 0 : st], *q1 = sm.q[1];
            float amax = 0.0f;
            uint32_t top = 0;
#pragma unroll 2
            for (int c = 0; c < D; c += 8) {
                const uint32_t off = tc::sw128_off(r, c, 128);
                const uint4 w = *reinterpret_cast<const uint4*>(q0 + off);
                if constexpr (F32) {
                    float x[8];
                    Vec16<T>::get(w, x);
                    Vec16<T>::get(*reinterpret_cast<const uint4*>(q1 + off), x + 4);
#pragma unroll
                    for (int d = 0; d < 8; ++d) amax = fmaxf(amax, fabsf(x[d]));
                } else {
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d) asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(v[d] & 0x7fff7fffu));
                }
            }
            if constexpr (!F32) amax = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
            const int eq = query_exponent(amax);
            const float f = exp2i(-eq);
#pragma unroll 2
            for (int c = 0; c < D; c += 8) {
                const uint32_t off = tc::sw128_off(r, c, 128);
                float x[8];
                uint32_t hi[4], lo[4];
                Vec16<T>::get(*reinterpret_cast<const uint4*>(q0 + off), x);
                if constexpr (F32) Vec16<T>::get(*reinterpret_cast<const uint4*>(q1 + off), x + 4);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float y0 = x[2 * d] * f, y1 = x[2 * d + 1] * f;
                    hi[d] = tc::pack_f16(y0, y1);
                    if constexpr (F32) {
                        const float2 b = tc::unpack_f16(hi[d]);
                        lo[d] = tc::pack_f16(y0 - b.x, y1 - b.y);
                    }
                }
                *reinterpret_cast<uint4*>(q0 + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if constexpr (F32) *reinterpret_cast<uint4*>(q1 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.qfull[st]));
            return p.scale2 * exp2i(eq);
        };
        // bf16: adds the row's sums to what has been set aside of them, if anything, where the row's partial result goes in the
        // end: there (keep), or in tensor memory.
        auto set_aside = [&](const Segment& s, float m, bool any, bool keep) {
            const long long row = (long long)(blockIdx.x * 2 + (s.first ? 1 : 0)) * kRows + tid;
            const float mf = any ? p.part_ml[row].x : 0.0f, f = mf == -INFINITY ? 0.0f : tc::ex2_approx(mf - m);
            float4* at = reinterpret_cast<float4*>(p.part_o + row * D);
#pragma unroll 1
            for (int c = 0; c < D; c += 16, at += 4) {
                float o[16];
                float4 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = any ? at[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                tc::tmem_ld16(tO + c, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[4 * i] = fmaf(y[i].x, f, o[4 * i]), o[4 * i + 1] = fmaf(y[i].y, f, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(y[i].z, f, o[4 * i + 2]), o[4 * i + 3] = fmaf(y[i].w, f, o[4 * i + 3]);
                }
                if (keep) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) at[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else {
                    uint32_t b[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(o[i]);
                    tc::tmem_st16(tO + c, b);
                }
            }
            if (keep) p.part_ml[row].x = m;
            else tc::tmem_st_wait();
        };
        // The segment's results: outputs of a whole item, a partial result otherwise.
        auto put = [&](const Segment& s, float m, float l) {
            const int row = s.twin ? r : tid, rr = s.rb * kRows + row, t = p.token_of(rr), hq = s.h * p.G + rr - t * p.G;
            const bool any = s.nt[st] > 0;
            if (!F32 && s.nt[st] > kFold) set_aside(s, m, true, false);
            // Twin streams: rows r of both lie in the same lanes of tensor memory, so that stream 0 reads both accumulators.
            const bool join = s.twin && s.nt[1] > 0;
            float f = 1.0f, f1 = 0.0f;  // of this stream's and the other one's part of the row
            if (join && st == 1) {
                sm.twin_ml[r] = make_float2(m, l);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.tfull));
                owed = true;  // stream 0's reading, before the next products of this stream
                return;
            }
            if (join) {
                ok = ok && tc::mbar_wait(tc::smem_u32(&sm.tfull), n_t++ & 1);
                tc::fence_after_sync();
                const float2 ml = sm.twin_ml[r];
                const float mm = fmaxf(m, ml.x);
                f = m == -INFINITY ? 0.0f : tc::ex2_approx(m - mm);
                f1 = ml.x == -INFINITY ? 0.0f : tc::ex2_approx(ml.x - mm);
                // a row that has seen nothing, or NaN, keeps m = -inf: its sum counts as it is
                l = (m == -INFINITY ? l : l * f) + (ml.x == -INFINITY ? ml.y : ml.y * f1);
                m = mm;
            }
            const bool mine = row < s.rows && !s.g.dead && !(s.twin && st == 1);
            const long long orow = (long long)(s.g.row0 + t) * p.HQ + hq;
            const bool complete = s.first && s.last;
            const long long slot = (long long)(blockIdx.x * 2 + (s.first ? 1 : 0)) * kRows + row;
            const float inv = complete ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            if (mine) {
                if (!complete) p.part_ml[slot] = make_float2(m, l);
                else if (p.lse) p.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
            if (any) {
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float o[16];
                    tc::tmem_ld16(tO + c, o);
                    tc::tmem_ld_wait();
                    if (!F32 && join) {
                        float other[16];
                        tc::tmem_ld16(tO + 128 + c, other);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], f, other[i] * f1);
                    }
                    if (F32 && s.nt[st] > kFold) {
                        float sum[16];
                        tc::tmem_ld16(tSum + c, sum);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] += sum[i];
                    }
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= inv;
                        const int half = c < 64 ? 0 : 8;  // see chunk_of
                        if (complete) {
#pragma unroll
                            for (int i = 0; i < 16; i += Vec16<T>::kN)
                                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + orow * D + c + (i ^ half)) = Vec16<T>::put(o + i);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<float4*>(p.part_o + slot * D + c + (i ^ half)) =
                                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                }
                tc::fence_before_sync();  // these reads come before the products that the next weights admit
                if (join) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.tempty));
                }
            }
        };
        const Segment* sp = nullptr;
        float m = 0.0f, l = 0.0f;
        while (true) {
            // the next segment's queries come while the last products of this one run
            const Segment* np = take();
            float rs_next = 0.0f;
            if (np && np->nt[st] > 0) rs_next = queries(*np);
            if (sp) {
                if (sp->nt[st] > 0) {
                    ok = ok && tc::mbar_wait(tc::smem_u32(&sm.ofull[st]), n_o & 1);
                    ++n_o;
                    tc::fence_after_sync();
                }
                if (ok) put(*sp, m, l);
                give(sp);
            }
            sp = np;
            if (!sp || !ok) break;
            const Segment& s = *sp;
            const int nt = s.nt[st];
            const float rs = rs_next;
            m = -INFINITY, l = 0.0f;
            if (s.g.dead) {
                if (tid < s.rows) {
                    const int rr = s.rb * kRows + tid, t = p.token_of(rr), hq = s.h * p.G + rr - t * p.G;
                    const long long orow = (long long)(s.g.row0 + t) * p.HQ + hq;
#pragma unroll
                    for (int c = 0; c < (int)(D * sizeof(T) / 16); ++c)
                        reinterpret_cast<uint4*>(static_cast<T*>(p.out) + orow * D)[c] = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[orow] = -INFINITY;
                }
                if (tid == 0 && s.g.bad_len) raise_error(p.hdr, GDN_DEVERR_KV_LEN);
                if (tid == 0 && s.bad_tree) raise_error(p.hdr, GDN_DEVERR_TREE);
            }
            if (tid == 0 && s.first && !s.last && !s.g.dead) meta = make_int4(s.n, s.h, s.rb, s.end_cta);
            if (nt > 0) {
                const Tree& tree = sm.tree[sp - sm.seg];
                const int ta = s.t.a, skip = s.t.b - ta, k0 = s.k0;
                const int row0 = s.twin ? 0 : st * 128, row = row0 + r;
                const bool mine = row < s.rows;
                const int rr = s.rb * kRows + row, t = mine ? p.token_of(rr) : 0, hq = s.h * p.G + (mine ? rr - t * p.G : 0);
                // the row sees tokens [vlo, vhi) and [0, pre)
                int pos = s.g.base + t;
                uint32_t anc = 0;  // of a tree: the row's draft and its ancestors
                if (p.parents) {
                    anc = tree.anc[t];
                    pos = s.g.base + __popc(anc) - 1;
                }
                const int vlo = p.window > 0 ? max(0, pos + 1 - p.window) : 0, vhi = mine ? pos + 1 : vlo, pre = mine ? s.t.pre : 0;
                const int r_first = s.rb * kRows + row0, r_last = s.rb * kRows + min(row0 + 127, s.rows - 1);
                // (every row sees the tokens up to pos_first: of a tree, not even the first draft)
                const int pos_first = s.g.base + (p.parents ? -1 : p.token_of(r_first)), pos_last = s.g.base + p.token_of(r_last);
                const float slope = p.slopes ? p.slopes[hq] * kLog2e : 0.0f;
                const float cap2 = p.cap2, cap_in = CAP != kNoCap ? 2.0f * kLog2e / cap2 : 0.0f;

                int j = 0;
                do {  // (a loop of its own for what is added up before it is set aside)
                    do {
                        const int i = s.twin ? 2 * j + st : j, k = k0 + i, t0 = (k < ta ? k : k + skip) * kTile, es = (tile + i) % kExpSlots;
                        ok = tc::mbar_wait(tc::smem_u32(&sm.sfull[st]), n_s & 1);
                        ++n_s;
                        tc::fence_after_sync();
                        // every row of the stream sees the whole tile, and no bias depends on the place
                        const bool whole = !p.slopes && ((t0 + kTile - 1 <= pos_first && (p.window <= 0 || pos_last - t0 < p.window)) ||
                                                         t0 + kTile <= s.t.pre);
                        const uint32_t scales = tc::smem_u32(sm.scale[es]);
                        // read where they are used, each time (kept in registers they would make the scores spill)
                        auto scale = [&](int g) {
                            float4 f;
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                                         : "r"(scales + g * 16));
                            f.x = fmaxf(1.0e-37f, fminf(rs * f.x, 3.0e38f));  // a masked score, -inf, stays that
                            return f;
                        };
                        const bool plain = CAP == kNoCap && !p.slopes;  // scores are only scaled, below; otherwise the scale below is 1
                        if (!whole) {
                            // Mask (unless plain: scale, cap and bias too) in tensor memory, 16 columns at a time, in loops of
                            // their own: unrolled over the registers below they would double the loop's code.
                            auto rewrite = [&](auto edit) {
#pragma unroll 1
                                for (int g = 0; g < kTile / 16; ++g) {
                                    float y[16];
                                    uint32_t b[16];
                                    tc::tmem_ld16(tS + g * 16, y);
                                    const float a = scale(g).x;
                                    tc::tmem_ld_wait();
                                    if constexpr (CAP != kNoCap) cap16<CAP>(y, a, cap2, cap_in);
                                    if (CAP == kNoCap && !plain)
#pragma unroll
                                        for (int i = 0; i < 16; ++i) y[i] *= a;
                                    edit(y, t0 + g * 16);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(y[i]);
                                    tc::tmem_st16(tS + g * 16, b);
                                }
                                tc::tmem_st_wait();
                            };
                            auto sees = [&](int tok) { return (uint32_t)(tok - vlo) < (uint32_t)(vhi - vlo) || tok < pre; };
                            auto biased = [&](float y, int at) { return fmaf(-slope, fabsf((float)(pos - at)), y); };
                            if (!p.slopes && !p.parents) {
                                rewrite([&](float* y, int tok) {
#pragma unroll
                                    for (int i = 0; i < 16; ++i) y[i] = sees(tok + i) ? y[i] : -INFINITY;
                                });
                            } else {
                                rewrite([&](float* y, int tok) {
                                    if (p.parents && tok + 16 > s.g.base && tok < s.g.kv) {  // drafts of a tree among the tokens
#pragma unroll
                                        for (int i = 0; i < 16; ++i) {
                                            const int d = max(0, min(tok + i - s.g.base, s.g.L - 1));
                                            const int at = tok + i < s.g.base ? tok + i : s.g.base + tree.depth[d];
                                            const bool seen = tok + i < s.g.base ? sees(tok + i)
                                                                                 : (((anc >> d) & 1) && at >= vlo && tok + i < s.g.kv) || tok + i < pre;
                                            y[i] = seen ? (p.slopes ? biased(y[i], at) : y[i]) : -INFINITY;
                                        }
                                    } else {
#pragma unroll
                                        for (int i = 0; i < 16; ++i)
                                            y[i] = sees(tok + i) ? (p.slopes ? biased(y[i], tok + i) : y[i]) : -INFINITY;
                                    }
                                });
                            }
                        }
                        float x[kTile];
#pragma unroll
                        for (int c = 0; c < kTile; c += 32) tmem_ld32(tS + c, x + c);
                        tc::tmem_ld_wait();
                        if constexpr (CAP != kNoCap) {  // scaled and capped here; below the scale is 1
                            if (whole)
#pragma unroll
                                for (int g = 0; g < kTile / 16; ++g) cap16<CAP>(x + g * 16, scale(g).x, cap2, cap_in);
                        }
                        float mx = -INFINITY;
#pragma unroll
                        for (int g = 0; g < kTile / 16; ++g) {
                            const float* y = x + g * 16;
                            const float m0 = max3(y[0], y[1], y[2]), m1 = max3(y[3], y[4], y[5]), m2 = max3(y[6], y[7], y[8]),
                                        m3 = max3(y[9], y[10], y[11]), m4 = max3(y[12], y[13], y[14]);
                            const float4 f = scale(g);
                            mx = fmaxf(mx, fmaf(fmaxf(max3(m0, m1, m2), max3(m3, m4, y[15])), plain ? f.x : 1.0f, f.y));
                        }
                        auto for_output = [&](uint32_t cols, float f) {  // scales 32 lanes of an accumulator
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                uint32_t b[16];
                                tc::tmem_ld16(cols + c, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(o[i] * f);
                                tc::tmem_st16(cols + c, b);
                            }
                        };
                        if constexpr (F32) {
                            if (j > 0 && j % kFold == 0) {  // the tensor core starts O anew at this tile
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    float o[16], sum[16];
                                    uint32_t b[16];
                                    tc::tmem_ld16(tO + c, o);
                                    tc::tmem_ld16(tSum + c, sum);
                                    tc::tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(j == kFold ? o[i] : o[i] + sum[i]);
                                    tc::tmem_st16(tSum + c, b);
                                }
                                tc::tmem_st_wait();
                            }
                        }
                        const bool move = mx > m + kMaxWeight;
                        if (__any_sync(0xffffffffu, move)) {
                            float fo = 1.0f;
                            if (move) {
                                fo = tc::ex2_approx(m - (mx - lift<F32>()));  // 0 from m = -inf
                                m = mx - lift<F32>();
                                l *= fo;
                            }
                            if (j % kFold != 0) for_output(tO, fo);
                            if (F32 && j >= kFold) for_output(tSum, fo);
                        }
                        if (owed) {
                            ok = ok && tc::mbar_wait(tc::smem_u32(&sm.tempty), n_t++ & 1);
                            owed = false;
                        }
                        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
                        for (int g = 0; g < kTile / 16; ++g) {
                            const float4 f = scale(g);
                            const float a = plain ? f.x : 1.0f, off = f.y - ref;
                            float* y = x + g * 16;
                            float s0 = 0.0f, s1 = 0.0f;
                            uint32_t hi[8], lo[8];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                fma2(y[i], y[i + 1], a, off);
                                y[i] = tc::ex2_approx(y[i]);
                                y[i + 1] = tc::ex2_approx(y[i + 1]);
                                add2(s0, s1, y[i], y[i + 1]);
                                hi[i / 2] = tc::pack_f16(y[i], y[i + 1]);
                                if constexpr (F32) {
                                    const float2 b = tc::unpack_f16(hi[i / 2]);
                                    lo[i / 2] = tc::pack_f16(y[i] - b.x, y[i + 1] - b.y);
                                }
                            }
                            l = fmaf(s0 + s1, f.z, l);
                            tc::tmem_st8(tP + g * 8, hi);  // in place of the scores (fp32: in the idle stream's columns)
                            if constexpr (F32) tc::tmem_st8(tP + 64 + g * 8, lo);
                        }
                        tc::tmem_st_wait();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.pfull[st]));
                    } while (++j < nt && ok && (F32 || j % kFold != 0));
                    if (!F32 && j < nt && ok) {  // with the next scores the products before them have completed
                        ok = tc::mbar_wait(tc::smem_u32(&sm.sfull[st]), n_s & 1);
                        tc::fence_after_sync();
                        set_aside(s, m, j > kFold, true);
                        tc::fence_before_sync();
                    }
                } while (j < nt && ok);
            }
            tile += s.steps;
        }
    } else if (warp < 12) {
        // ---------------- codes to operand tiles.  Eight lanes read 128 consecutive bytes, and write eight chunks of 8
        // fp16 that lie in different banks (see chunk_of; at D = 64 the swizzle of two rows sees to it).
        const int pt = (warp - 8) * 32 + lane;
        constexpr int kPerRow = D / 16, kIters = kTile * kPerRow / 128;
        const int c = pt % kPerRow, r0 = pt / kPerRow;  // 16-code chunk; rows r0, r0 + 128 / kPerRow, ...
        auto widen_tile = [&](int kv, uint8_t* dst, auto live) {
            const uint8_t* src = sm.raw[kv] + pt * 16;
#pragma unroll 1
            for (int i = 0; i < kIters; ++i) {
                const int r = r0 + i * (128 / kPerRow);
                uint4 raw = *reinterpret_cast<const uint4*>(src + i * 2048), lo, hi;
                if (!live(r)) raw = make_uint4(0, 0, 0, 0);
                widen16(raw, lo, hi);
                const uint32_t at = tc::sw128_off(r, chunk_of(2 * c) * 8, kTile);
                *reinterpret_cast<uint4*>(dst + at) = lo;
                *reinterpret_cast<uint4*>(dst + (at ^ 16u)) = hi;
            }
            tc::fence_smem_to_async();
            __syncwarp();
        };
        for (const Segment* sp = take(); sp && ok; give(sp), sp = take()) {
            const Segment& s = *sp;
            const int steps = s.steps;
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t g = tile + j, sg = g & 1, ph = (g >> 1) & 1;
                // the stage is free once the products of two tiles ago have completed
                ok = tc::mbar_wait(tc::smem_u32(&sm.rfull[0]), g & 1) && tc::mbar_wait(tc::smem_u32(&sm.kempty[sg]), ph ^ 1);
                widen_tile(0, sm.k[sg], [](int) { return true; });
                if (lane == 0) {
                    tc::mbar_arrive(tc::smem_u32(&sm.rempty[0]));
                    tc::mbar_arrive(tc::smem_u32(&sm.kfull[sg]));
                }
                ok = ok && tc::mbar_wait(tc::smem_u32(&sm.rfull[1]), g & 1) &&
                     tc::mbar_wait(tc::smem_u32(&sm.vempty[sg]), ph ^ 1);
                // values that no row sees have weight zero, but may be NaN codes
                const int k = s.k0 + j, t0 = (k < s.t.a ? k : k + s.t.b - s.t.a) * kTile;
                if ((t0 >= s.t.lo && t0 + kTile <= s.g.kv) || t0 + kTile <= s.t.pre)
                    widen_tile(1, sm.v[sg], [](int) { return true; });
                else
                    widen_tile(1, sm.v[sg],
                               [&](int r) { return (t0 + r >= s.t.lo && t0 + r < s.g.kv) || t0 + r < s.t.pre; });
                if (lane == 0) {
                    tc::mbar_arrive(tc::smem_u32(&sm.rempty[1]));
                    tc::mbar_arrive(tc::smem_u32(&sm.vfull[sg]));
                }
            }
            tile += steps;
        }
    } else if (warp == 12) {
        // ---------------- copies: lane g takes 16-token group g of a tile (a group lies within a page); page and
        // exponents are looked up a tile ahead
        const int ps_mask = (1 << p.ps_shift) - 1;
        uint32_t issued[2] = {0, 0};
        for (const Segment* sp = take(); sp && ok; give(sp), sp = take()) {
            const Segment& s = *sp;
            const int steps = s.steps;
            const int lo = s.t.lo, pre = s.t.pre, kv = s.g.kv, ta = s.t.a, skip = s.t.b - ta, k0 = s.k0, h = s.h;
            const int32_t* table = p.table + (long long)s.n * p.max_pages;
            int t = 0, pg = -1, ek = 0, ev = 0;
            // With few rows each key comes from HBM, and one tile's copies in flight would not cover its latency: twin
            // segments have the tiles kAhead further on brought to L2.
            constexpr int kAhead = 6;
            const bool ahead = s.twin;
            int t_far = 0, pg_far = -1;
            auto bring = [&](int j) {
                if (pg_far >= 0 && pg_far < p.num_pages) {
                    const long long o = ((((long long)pg_far * p.HKV + h) << p.ps_shift) + (t_far & ps_mask)) * D;
                    tc::bulk_prefetch_l2(p.k + o, 16 * D);
                    tc::bulk_prefetch_l2(p.v + o, 16 * D);
                }
                pg_far = -1;
                if (j < steps && lane < kTile / 16) {
                    t_far = (k0 + j < ta ? k0 + j : k0 + j + skip) * kTile + lane * 16;
                    if (t_far < pre || (t_far < kv && t_far + 15 >= lo)) pg_far = __ldg(table + (t_far >> p.ps_shift));
                }
            };
            auto look = [&](int j) {  // where no row sees a token of the group nothing is looked up
                t = (k0 + j < ta ? k0 + j : k0 + j + skip) * kTile + lane * 16;
                pg = -1;
                if (lane < kTile / 16 && (t < pre || (t < kv && t + 15 >= lo))) {
                    pg = __ldg(table + (t >> p.ps_shift));
                    if (pg < 0 || pg >= p.num_pages) {
                        raise_error(p.hdr, GDN_DEVERR_PAGE_RANGE);
                        pg = -1;
                    }
                }
                ek = pg >= 0 ? (int)__ldg(p.k_exp + (long long)pg * p.HKV + h) : 0;
                ev = pg >= 0 ? (int)__ldg(p.v_exp + (long long)pg * p.HKV + h) : 0;
            };
            if (steps > 0) look(0);
            if (ahead)
                for (int j = 1; j <= kAhead; ++j) bring(j);
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t g = tile + j;
                const long long off = ((((long long)max(pg, 0) * p.HKV + h) << p.ps_shift) + (t & ps_mask)) * D;
                const bool have = pg >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, have)) * 16u * D;
                if (lane < kTile / 16)
                    sm.scale[g % kExpSlots][lane] = make_float4(exp2i(ek), (float)ev, exp2i(-ev), 0.0f);
                __syncwarp();  // lane 0's arrival below passes them on
                if (j + 1 < steps) look(j + 1);
                if (ahead) bring(j + kAhead + 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // free once the tile before has been widened
                    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(tc::smem_u32(&sm.rempty[i]), (g & 1) ^ 1));
                    if (ok && lane == 0) tc::mbar_expect_tx(tc::smem_u32(&sm.rfull[i]), bytes);
                    __syncwarp();
                    if (ok && have)
                        tc::bulk_g2s(tc::smem_u32(sm.raw[i]) + lane * 16 * D, (i ? p.v : p.k) + off, 16 * D,
                                     tc::smem_u32(&sm.rfull[i]));
                    issued[i] += ok;
                }
            }
            tile += steps;
        }
        if (!ok)  // copies in flight land before the block ends
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (issued[i]) tc::mbar_wait(tc::smem_u32(&sm.rfull[i]), (issued[i] - 1) & 1, 100000000ull);
    } else if (warp == 15) {
        // ---------------- products (the whole warp walks and waits; one lane issues)
        const uint32_t q_s = tc::smem_u32(sm.q[0]);
        uint32_t phases = 0;  // of qfull (bits 0, 1) and pfull (bits 2, 3)
        // Descriptors are a base and a constant per k-step.  The bases pass through an empty asm so that they are
        // formed anew (an addition each) where the compiler would keep dozens of them, spilled, for the whole loop.
        const uint64_t q_d = tc::make_desc_sw128(q_s, 16, 1024), k_d = tc::make_desc_sw128(tc::smem_u32(sm.k[0]), 16, 1024),
                       v_d = tc::make_desc_sw128(tc::smem_u32(sm.v[0]), kTile * 128, 1024);
        auto anew = [](uint64_t d) {
            asm volatile("" : "+l"(d));
            return d;
        };
        auto scores = [&](int st, uint32_t sg) {  // S = Q K^T of a stream
            const uint64_t kd = anew(tc::desc_add(k_d, sg * (uint32_t)sizeof(sm.k[0])));
#pragma unroll
            for (int part = 0; part < (F32 ? 2 : 1); ++part) {
                const uint64_t qd = anew(tc::desc_add(q_d, (F32 ? part : st) * (uint32_t)sizeof(sm.q[0])));
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
                    tc::mma_f16(tm + st * 128, tc::desc_add(qd, tc::sw128_kstep(128, k)),
                                tc::desc_add(kd, tc::sw128_kstep(kTile, k)), kIdS, part > 0 || k > 0);
            }
            tc::mma_commit(tc::smem_u32(&sm.sfull[st]));
            tc::mbar_arrive(tc::smem_u32(&sm.sfull[st]));  // passes on the exponents that came with the keys
        };
        auto values = [&](int st, uint32_t sg, bool add) {  // O += P V
            const uint64_t vd = anew(tc::desc_add(v_d, sg * (uint32_t)sizeof(sm.v[0])));
#pragma unroll
            for (int part = 0; part < (F32 ? 2 : 1); ++part)
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc::mma_f16_ta(tm + 256 + st * 128, tm + (F32 ? 128 + part * 64 : st * 128) + k * 8,
                                   tc::desc_add(vd, k * 2048), kIdO, add || part > 0 || k > 0);
        };
        for (const Segment* sp = take(); sp && ok; give(sp), sp = take()) {
            // (broadcast, so that the compiler knows the descriptors to be the same in all lanes)
            const int nt0 = __shfl_sync(0xffffffffu, sp->nt[0], 0), nt1 = __shfl_sync(0xffffffffu, sp->nt[1], 0);
            const int twin = __shfl_sync(0xffffffffu, (int)sp->twin, 0), steps = max(nt0, nt1);
            // step j: the weights of a stream's tile j times its values, then the scores of its tile j + 1, one stream after
            // the other.  Both streams' tile j is tile j of the segment, or (twin) tiles 2 j and 2 j + 1.
            for (int j = -1; j < steps && ok; ++j) {
#pragma unroll 1
                for (int st = 0; st < 2; ++st) {
                    const int nt = st ? nt1 : nt0;
                    if (!ok || j >= nt || nt == 0) continue;
                    const uint32_t g = tile + (twin ? 2 * j + st : j), g1 = twin ? g + 2 : g + 1;
                    const bool pv = j >= 0, qk = j + 1 < nt, last = twin || st == 1 || j >= nt1;  // the tile's last use
                    if (pv) ok = tc::mbar_wait(tc::smem_u32(&sm.vfull[g & 1]), (g >> 1) & 1);
                    if (qk) ok = ok && tc::mbar_wait(tc::smem_u32(&sm.kfull[g1 & 1]), (g1 >> 1) & 1);
                    // the stream's queries (of this segment), or its weights (of tile j)
                    const uint32_t bar = pv ? tc::smem_u32(&sm.pfull[st]) : tc::smem_u32(&sm.qfull[st]);
                    const uint32_t bit = (pv ? 4u : 1u) << st;
                    ok = ok && tc::mbar_wait(bar, (phases & bit) != 0);
                    phases ^= bit;
                    if (!ok) continue;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        if (pv) {
                            values(st, g & 1, j % kFold != 0);
                            if (last) tc::mma_commit(tc::smem_u32(&sm.vempty[g & 1]));
                        }
                        if (qk) {
                            scores(st, g1 & 1);
                            if (twin || st == 1 || j + 1 >= nt1) tc::mma_commit(tc::smem_u32(&sm.kempty[g1 & 1]));
                            if (j + 2 >= nt) tc::mma_commit(tc::smem_u32(&sm.qempty[st]));
                        } else {
                            tc::mma_commit(tc::smem_u32(&sm.ofull[st]));
                        }
                    }
                    __syncwarp();
                }
            }
            tile += sp->steps;
        }
    } else if (warp == 14) {
        // ---------------- queries: rows as they are, to where their stream converts them, once the products with the queries
        // before them have completed.  Asynchronous 16-byte copies; neighbouring lanes take neighbouring chunks of a row.
        constexpr int kLanes = D * (int)sizeof(T) / 16, kRowsEach = 32 / kLanes;
        const int c = lane % kLanes;
        // fp32: dimensions 8 i .. 8 i + 3 to the first tile, the next four to the second, at the place of their 8 results
        const int place = chunk_of(F32 ? c >> 1 : c) * 8, side = F32 ? c & 1 : 0;
        const int head_step = kRowsEach % p.G;
        const long long step = (long long)(kRowsEach / p.G) * p.q_stride + head_step * D, wrap = p.q_stride - (long long)p.G * D;
        uint32_t phases = 0;
        for (const Segment* sp = take(); sp && ok; give(sp), sp = take()) {
            const Segment& s = *sp;
#pragma unroll 1
            for (int st = 0; st < 2; ++st) {
                if (s.nt[st] == 0) continue;
                ok = ok && tc::mbar_wait(tc::smem_u32(&sm.qempty[st]), ((phases >> st) & 1) ^ 1);
                if (!ok) break;
                phases ^= 1u << st;
                const uint32_t dst = tc::smem_u32(sm.q[F32 ? side : st]);
                // rows go up by kRowsEach: (token, head of the group) and the address follow by additions
                const int first = (s.twin ? 0 : st * 128) + lane / kLanes, rr = s.rb * kRows + first, t = p.token_of(rr);
                int left = s.rows - first, head = rr - t * p.G;
                const T* src = static_cast<const T*>(p.q) + (long long)(s.g.row0 + t) * p.q_stride + (long long)(s.h * p.G + head) * D +
                               c * (16 / (int)sizeof(T));
#pragma unroll 1
                for (int i0 = 0; i0 < 128; i0 += 4 * kRowsEach) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = i0 + j * kRowsEach + lane / kLanes;
                        copy16_or_zero(dst + tc::sw128_off(i, place, 128), left > 0 ? src : static_cast<const T*>(p.q), left > 0);
                        left -= kRowsEach;
                        head += head_step;
                        src += step;
                        if (head >= p.G) head -= p.G, src += wrap;
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&sm.qraw[st])) : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 13) {
        // ---------------- the segments, a few ahead of their use
        Walk<kRows, !F32> w;
        bool more = w.begin(p);
        for (uint32_t n = 0; ok; ++n) {
            const uint32_t at = n % kSegSlots;
            Segment s;
            more = more && w.next(p, s);
            ok = tc::mbar_wait(tc::smem_u32(&sm.segempty[at]), ((n / kSegSlots) & 1) ^ 1);
            if (ok && more && p.parents && lane < kMaxVerifyDraft) {
                sm.tree[at].anc[lane] = (uint16_t)w.anc;
                sm.tree[at].depth[lane] = (int8_t)(__popc(w.anc) - 1);
            }
            if (ok && lane == 0) {
                if (more) sm.seg[at] = s;
                sm.more[at] = more;
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(tc::smem_u32(&sm.segfull[at]));
            if (!more) break;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {
        if (tid == 0) raise_error(p.hdr, GDN_DEVERR_TIMEOUT);
        if (tid == 15 * 32) {  // products still in flight finish before the tensor memory is released
            tc::mma_commit(tc::smem_u32(&sm.drained));
            tc::mbar_wait(tc::smem_u32(&sm.drained), 0, 100000000ull);
        }
        __syncthreads();
    }
    if (tid == 0) p.meta[blockIdx.x] = ok ? meta : make_int4(-1, 0, 0, 0);
    if (warp == 0) tc::tmem_dealloc(sm.tmem, 512);
}

// Joins the partial results of the item that begins in CTA blockIdx.x and goes on in others, in the order of
// its tiles: a warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_rows_kernel(const __grid_constant__ Args p, int item_rows) {
    wait_for_launch_before();
    const int4 meta = p.meta[blockIdx.x];
    if (meta.x < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Geometry g = geometry(p, meta.x);
    const int first = blockIdx.x, count = meta.w - first + 1;
    constexpr int kCols = D / 32;
    for (int row = blockIdx.y * 8 + warp; row < item_rows; row += gridDim.y * 8) {
        const int rr = meta.z * item_rows + row;
        if (rr >= g.L * p.G) return;
        auto slot = [&](int i) { return (long long)((first + i) * 2 + (i == 0 ? 1 : 0)) * item_rows + row; };
        float mm = -INFINITY;
        for (int i = lane; i < count; i += 32) mm = fmaxf(mm, p.part_ml[slot(i)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        float l = 0.0f, x[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) x[c] = 0.0f;
        for (int i = 0; i < count; ++i) {
            const float2 ml = p.part_ml[slot(i)];
            if (ml.x == -INFINITY) {  // this part saw nothing (or a NaN: it is in the sum)
                l += ml.y;
                continue;
            }
            const float f = tc::ex2_approx(ml.x - mm);
            l = fmaf(ml.y, f, l);
#pragma unroll
            for (int c = 0; c < kCols; c += 2) {
                const float2 y = reinterpret_cast<const float2*>(p.part_o + slot(i) * D)[lane + c * 16];
                x[c] = fmaf(f, y.x, x[c]);
                x[c + 1] = fmaf(f, y.y, x[c + 1]);
            }
        }
        const int t = p.token_of(rr), hq = meta.y * p.G + rr - t * p.G;
        const long long orow = (long long)(g.row0 + t) * p.HQ + hq;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
            T* at = static_cast<T*>(p.out) + orow * D + 2 * lane + c * 32;
            at[0] = from_f<T>(x[c] * inv);
            at[1] = from_f<T>(x[c + 1] * inv);
        }
        if (p.lse && lane == 0) p.lse[orow] = l == 0.0f ? -INFINITY : (mm + log2f(l)) * kLn2;
    }
}

template <typename T, int D, Cap CAP>
cudaError_t launch(const Args& p, cudaStream_t s) {
    constexpr int kRows = item_rows<sizeof(T) == 4>();
    const int smem = (int)sizeof(Smem<D, kRows>);
    static_assert(sizeof(Smem<D, kRows>) <= 227 * 1024, "more shared memory than a block can have");
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(extend_kernel<T, D, CAP>), smem, done);
    if (e != cudaSuccess) return e;
    plan_kernel<<<1, 1024, 0, s>>>(p, kRows);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_after(extend_kernel<T, D, CAP>, dim3(kGrid), kThreads, smem, s, p)) != cudaSuccess) return e;
    return launch_after(join_rows_kernel<T, D>, dim3(kGrid, kRows / 16), 256, 0, s, p, kRows);
}

template <typename T, int D>
cudaError_t launch_dim(const Args& p, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    const Cap cap = cap_form<F32>(p.cap2);
    if (cap == kNoCap) return launch<T, D, kNoCap>(p, s);
    if constexpr (!F32)
        if (cap == kExpCap) return launch<T, D, kExpCap>(p, s);
    return launch<T, D, kTanhCap>(p, s);
}

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

// items of a batch: a row tile per item_rows rows, and one begun by each request
size_t max_items(int rows, long long N, long long TG) { return (size_t)(TG / rows + N); }

// Lays the workspace out behind the header; returns its end.
size_t carve(Args& p, int D, int rows, long long N, long long TG) {
    size_t at = kHeaderBytes;
    uint8_t* w = reinterpret_cast<uint8_t*>(p.hdr);
    auto take = [&](size_t bytes) {
        uint8_t* q = w ? w + at : nullptr;
        at += round16(bytes);
        return q;
    };
    const size_t items = max_items(rows, N, TG);
    p.plan = reinterpret_cast<int*>(take(16));
    p.items = reinterpret_cast<int2*>(take(items * sizeof(int2)));
    p.prefix_units = reinterpret_cast<long long*>(take((items + 1) * sizeof(long long)));
    p.meta = reinterpret_cast<int4*>(take(kGrid * sizeof(int4)));
    p.part_ml = reinterpret_cast<float2*>(take((size_t)2 * kGrid * rows * sizeof(float2)));
    p.part_o = reinterpret_cast<float*>(take((size_t)2 * kGrid * rows * D * sizeof(float)));
    return at;
}

int rows_of(int dtype) { return dtype == GDN_DTYPE_F32 ? item_rows<true>() : item_rows<false>(); }

}  // namespace

size_t extend_workspace_bytes(int D, int dtype, long long N, long long TG) {
    Args p{};
    return carve(p, D, rows_of(dtype), N, TG);
}

cudaError_t launch_extend_tc(Args p, int D, int dtype, cudaStream_t s) {
    carve(p, D, rows_of(dtype), p.N, (long long)p.T * p.G);
    if (dtype == GDN_DTYPE_F32) return D == 128 ? launch_dim<float, 128>(p, s) : launch_dim<float, 64>(p, s);
    return D == 128 ? launch_dim<__nv_bfloat16, 128>(p, s) : launch_dim<__nv_bfloat16, 64>(p, s);
}

}  // namespace attn
}  // namespace gdn
