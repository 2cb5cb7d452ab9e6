// Internal declarations of the 8-bit paged attention (include/attn.h).
#pragma once

#include <atomic>

#include "../../include/attn.h"
#include "gdn_internal.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 148;  // grid sizes and workspaces are made for B200's SM count; any other count is correct too

// One call's arguments.  Request n has L_n new rows; its "rows" below are (new row, query head of the
// group) pairs of one key/value head, G per new row, so that all of them read a key once.
struct Args {
    int HQ, HKV, G;
    uint32_t g_inv;  // ceil(2^32 / G), 0 for G = 1
    int ps_shift;  // log2(page_size)
    int window;    // <= 0: none
    float scale2;  // scale * log2(e): scores are kept in base-2 units
    float cap2;    // logit_cap * log2(e) within 2^-100 .. 2^120, 0: none
    const void* q;
    long long q_stride;
    const int32_t* cu;       // [N+1], or null: `per` rows each
    int per, N, T;
    int rows_above, rows_upto;  // the requests with rows_above < rows (per key/value head) <= rows_upto are this launch's
    const int32_t* kv_lens;  // [N]
    const int32_t* table;    // [N, max_pages]
    int max_pages;
    const uint8_t* k;
    const uint8_t* v;
    const int8_t* k_exp;
    const int8_t* v_exp;
    int num_pages;
    const float* slopes;       // nullable
    const int32_t* prefix;     // nullable
    const int32_t* parents;    // nullable: [N, per]
    void* out;
    float* lse;                // nullable
    int32_t* hdr;
    // workspace carve-out
    int* plan;                // attn_extend_tc.cu: the number of items,
    int2* items;              //   (request, row tile) of each,
    long long* prefix_units;  //   and the units before each and in all
    int4* meta;     // [grid]: the item (request, head, row block, last CTA) that begins in a CTA and goes on; -1: none
    float2* part_ml;  // [grid, 2, rows]: reference exponent and sum of a partial result
    float* part_o;    // [grid, 2, rows, head_dim]

    // row / G for rows below 2^25: with e = G * g_inv - 2^32 < G <= 128, row * e < 2^32, so the quotient is exact
    __device__ __forceinline__ int token_of(int row) const { return g_inv ? (int)__umulhi((uint32_t)row, g_inv) : row; }
};

struct AppendArgs {
    int HKV, ps_shift;
    const void* x[2];        // k_new, v_new
    long long stride[2];
    uint8_t* codes[2];
    int8_t* exps[2];
    const int32_t* cu;       // nullable: `per` rows each
    int per, N, T;
    const int32_t* start;
    const int32_t* table;
    int max_pages, num_pages;
    int32_t* hdr;
};

// The tokens that some row of a request sees: [0, pre) and [lo, kv).  (lo <= pre is folded to lo = 0.)
struct Range {
    int kv, lo, pre;
};

__device__ __forceinline__ Range visible_range(const Args& p, int n, int kv, int L) {
    Range r{kv, 0, 0};
    if (p.window > 0) r.lo = max(0, kv - L + 1 - p.window);
    if (r.lo > 0 && p.prefix) {
        r.pre = max(0, min(p.prefix[n], kv));
        if (r.pre >= r.lo) r.lo = r.pre = 0;
    }
    return r;
}

// The running reference m of a row's softmax, in base-2 units: set so that the largest weight 2^(s - m) is
// 2^lift, moved when one would exceed 2^kMaxWeight (46341 of fp16's 65504).  fp16 holds a weight with all its bits down to
// 2^-14 and to within 2^-25 below.  Moving costs a pass over the output, so bf16 starts low and leaves room for growth
// by 2^15.5 (weights off by at most 2^-25 of the largest).  fp32 keeps them to 2^-37 with room for 2^3.5: over
// 57426 tokens with scores far apart, 2^-31 left an error of 5.9e-6 where plain fp32 has 2e-6.
constexpr float kMaxWeight = 15.5f;
template <bool F32> __host__ __device__ constexpr float lift() { return F32 ? 12.0f : 0.0f; }

// 2^e for e in -126 .. 127
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The exponent eq for which |x| <= amax times 2^-eq lies below 2^14 in fp16: a row of queries keeps all
// of a bf16 value's bits down to 2^-28 of its largest.  The lower limit keeps 2^-eq within exp2i's range (values below
// 2^-113 need no more: bf16's smallest is 2^-133); the largest values need no limit (2^127: 114, inf: 115).
__device__ __forceinline__ int query_exponent(float amax) {
    return max(-126, (__float_as_int(amax) >> 23) - 127 - 13);  // amax >= 0; inf: 115
}

template <typename T> struct Vec16;  // 16 bytes of a row
template <> struct Vec16<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void get(uint4 w, float* x) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 put(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void get(uint4 w, float* x) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(v[i] << 16), x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ uint4 put(const float* x) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            v[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
};

// two e4m3 codes (the low and the high half of a word) as two fp16
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// 16-byte asynchronous copy, or 16 zero bytes
__device__ __forceinline__ void copy16_or_zero(uint32_t sdst, const void* gsrc, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sdst), "l"(gsrc), "r"(live ? 16 : 0)
                 : "memory");
}

// Lets a kernel take `bytes` of dynamic shared memory, once per device (`done`: a static word of the caller, a bit per device).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A kernel launched by launch_after starts while the launch before it on the stream still runs; it calls this before it
// reads what that one writes.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... A, typename... B>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t s, B... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<A>(args)...);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The two forms of cap * tanh(x / cap), in base-2 units.  kExpCap: cap - 2 cap / (1 + e^(2 x / cap)), cap_in =
// 2 log2(e) / cap; it is off by up to 2^-20 of the cap however small the score, so it serves bf16 alone, up to kMaxExpCap,
// where that is less than the weights' rounding to fp16.  kTanhCap: the library's tanh, off by 2^-20 of the score
// whatever the cap, for fp32 and for larger caps.  Caps 256 and 257 (B200): 12373 rows in a window, 16/4 heads of 128, 328
// and 535 us; 32 rows per key (64 requests of 500 to 8000 tokens, 8 key heads) 201 and 263 us; 8 rows per key 96 and 97 us.
enum Cap { kNoCap, kExpCap, kTanhCap };
constexpr float kMaxExpCap = 256.0f * kLog2e;
template <bool F32> inline Cap cap_form(float cap2) {
    return !(cap2 > 0.0f) ? kNoCap : F32 || cap2 > kMaxExpCap ? kTanhCap : kExpCap;
}
template <Cap CAP> __device__ __forceinline__ float capped(float x, float cap2, float cap_in) {
    if constexpr (CAP == kTanhCap) return cap2 * tanhf(__fdividef(x, cap2));
    else return cap2 - __fdividef(2.0f * cap2, 1.0f + tc::ex2_approx(x * cap_in));
}

cudaError_t launch_append(const AppendArgs& a, int head_dim, int dtype, cudaStream_t s);

// The rows per key up to which the split kernel is the faster one.  The kernel of 128-row tensor-core tiles takes the same time
// for 8 rows per key as for 128; the split kernel reads the cache once for every 32 rows, and fp32 at D = 128, two parts
// of each operand, falls behind with the last 16 of them.  Measured (B200, us, split / tiles; 64 requests of 500 to 8000
// tokens, 32/8 heads of 128): 8 rows per key 77 / 207, 16: 93 / 209, 24: 168 / 210, 32: 179 / 209, 40: 292 / 211, 48: 298 /
// 210; 2 key heads, 16 to 48 rows: 59, 101, 107, 164, 165 / 104 to 107; heads of 64, 32 and 40 rows: 109, 177 / 173.
// fp32, 16, 20, 32 and 40 rows: 118, 362, 374, 693 / 302 to 305; heads of 64: 83, 166, 173, 311 / 245.
constexpr int split_rows(int D, bool F32) { return F32 && D == 128 ? 16 : 32; }

// Attention over the cache, split along the tokens (attn_split.cu): any mode, few rows per key.
cudaError_t launch_split(Args a, int head_dim, int dtype, cudaStream_t s);
size_t split_workspace_bytes(int head_dim);

// Attention of many new rows on the tcgen05 tensor cores (attn_extend_tc.cu); rows: T * G.
cudaError_t launch_extend_tc(Args a, int head_dim, int dtype, cudaStream_t s);
size_t extend_workspace_bytes(int head_dim, int dtype, long long N, long long rows);

}  // namespace attn
}  // namespace gdn
