// The whole layer for a few tokens (T <= 16) in one persistent kernel.
//
// Decoding a few tokens is bound by the bytes of the experts they reach, so
// the kernel is a stream of weight rows through every SM that nothing
// interrupts: a producer warp loads 128-byte-wide pieces of weight rows by TMA
// into a ring in shared memory, and eight consumer warps multiply them with
// mma.sync (weights as the 16-row operand, tokens as the 8 columns; tcgen05's
// 128-row tiles would leave most SMs without a tile, and the few tokens cost
// nothing extra on the 8-column shape).  One block per SM, launched
// cooperatively; the phases are separated by grid barriers, and since weights
// do not depend on what the barriers wait for, the ring keeps filling across
// them:
//   1  router logits: (expert, slice of d) dot products in fp32, partial sums
//      per slice; x into the operand form of the weights' type;
//   -- barrier; every block then selects the top-K of all tokens for itself
//      (slices added in order), builds the list of experts reached, and takes
//      an equal share of their rows, 16 at a time:
//   2  h = SiLU(W1 x + b1), written per (token, slot);
//   -- barrier; FP8 and MXFP4: h into the operand form, barrier;
//   3  an equal share of the output rows: sum over the experts of
//      gate * (W2 h + b2), shared experts included, written once as bf16.
// The eight warps split K; their accumulators are added in warp order through
// shared memory, once per job in phase 2 and once in phase 3.  Columns are the
// tokens themselves: a token that did not choose the expert has a zero column.
//
// Operand forms (the products inside an MMA are exact, sums fp32):
//   bf16   weights, x and h in bf16;
//   FP8    e4m3 codes converted to fp16 (exact); x and h quantised to e4m3 per
//          128 columns, scales applied in fp32 per 64 columns of K;
//   MXFP4  E2M1 codes converted to fp16 (exact), the weight scale applied in
//          fp32 per block of 32; x and h in fp16 with a power-of-two scale per
//          128 columns, which brings their largest magnitude to 2^14..2^15:
//          bf16 values stay exact down to 2^-29 of it, and h keeps 11 bits.
// Every wait is bounded (common.cuh); after a wait gives up, the warps skip
// the remaining work but keep meeting at the block's barriers.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cstring>
#include "internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int CW = 8;                          // consumer warps
constexpr int CT = CW * 32;                    // consumer threads
constexpr int THREADS = CT + 32;               // + the producer warp
constexpr int SLOTS = 10, SLOT_BYTES = 16384;  // ring
constexpr int SCALE_BYTES = 1024;              // MXFP4: 8 scale bytes for each row of a slot
constexpr int RED_PITCH = 132;                 // floats per column of the reduction buffer (bank spread)
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;

constexpr int OFF_RING = 0;
constexpr int OFF_SCALES = OFF_RING + SLOTS * SLOT_BYTES;
constexpr int OFF_RED = OFF_SCALES + SLOTS * SCALE_BYTES;
constexpr int OFF_IDX = OFF_RED + CW * 8 * RED_PITCH * 4;      // [16][16] int
constexpr int OFF_GATE = OFF_IDX + MAX_T * 16 * 4;             // [16][16] float
constexpr int OFF_MASK = OFF_GATE + MAX_T * 16 * 4;            // [256] tokens kept, per expert
constexpr int OFF_KPACK = OFF_MASK + 256 * 4;                  // [256] 4 bits per token: its slot
constexpr int OFF_ACT = OFF_KPACK + 256 * 8;                   // [256] experts reached, ascending
constexpr int OFF_BAR = OFF_ACT + 256 * 4;                     // full, empty [SLOTS]
constexpr int OFF_MISC = OFF_BAR + 2 * SLOTS * 8;              // abort flag, n_active, 8 warp counts
constexpr int SMEM_BYTES = OFF_MISC + 64;
constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
static_assert(OFF_KPACK % 8 == 0 && OFF_BAR % 8 == 0 && OFF_RED % 16 == 0, "alignment");
static_assert(CW * 8 * RED_PITCH * 4 >= MAX_T * 256 * 4 + 256 * 4, "the router's probabilities fit the buffer");

// grid-wide counters in the workspace, zero between launches
enum { CTR_BAR = 0, CTR_EXIT = 3, CTR_ABORT = 4, CTR_WORDS = 5 };

struct __align__(64) FewParams {
    CUtensorMap w1, w2, ws1, ws2;
    const __nv_bfloat16* x;
    const float* W_r;
    const float* logit_bias;      // added to the logits, or nullptr
    const float* sel_bias;        // added to the selection keys, or nullptr
    const void *w1s, *w2s, *ws1s, *ws2s;
    const float *b1, *b2, *bs1, *bs2;
    __nv_bfloat16* out;
    float *f, *P, *loss;
    int32_t *topk_idx, *counts;   // or nullptr
    float* gates;                 // or nullptr
    // workspace
    int32_t* status;
    uint32_t* ctr;
    float* part;                  // (ks, T, E) partial logits
    uint8_t* xq;                  // x in operand form (bf16: x itself)
    float* xs;                    // (T, d / 128) its scales
    float* h32;                   // fp32 h: (T K, dff), then (S T, dffs)
    uint8_t* hq;                  // h in operand form, same rows
    float* hs;                    // its scales per 128
    float alpha;
    int T, d, E, K, dff, S, dffs, capacity, slot_major, passthrough;
    int ks, slice;                // router slices of d and their length
    int rows3;                    // output rows of a phase-3 job (the W2 maps' box)
};

enum { M_BF16 = 0, M_FP8 = 1, M_FP4 = 2 };

template <int MODE> struct Form;
// K elements in 64 bytes of a weight row (a warp's half of a 128-byte piece);
// bytes of an operand element of x and h
template <> struct Form<M_BF16> { static constexpr int KH = 32, BB = 2; };
template <> struct Form<M_FP8> { static constexpr int KH = 64, BB = 1; };
template <> struct Form<M_FP4> { static constexpr int KH = 128, BB = 2; };

__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" :: "n"(CT) : "memory"); }

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(smem_u32(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

// Arrives on bar once this thread's earlier cp.async copies have landed (the
// barrier's count includes the arrival).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes to two pairs of fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}

// ---------------------------------------------------------------- operand form of x and h

// 128 values, four per lane, into the operand form: codes and one scale.
template <int MODE>
__device__ __forceinline__ void store_block(const float (&v)[4], uint8_t* dst, float* scale, int lane) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xffffffffu, m);
    if (MODE == M_FP8) {
        // fmaxf semantics of the dispatch quantiser: a NaN does not count
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = fmaxf(a, fabsf(v[j]));
        m = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
        const float sc = pow2_scale_448(__uint_as_float(m)), inv = inv_pow2(sc);
        const uint32_t lo = f32x2_to_e4m3x2(v[0] * inv, v[1] * inv), hi = f32x2_to_e4m3x2(v[2] * inv, v[3] * inv);
        reinterpret_cast<uint32_t*>(dst)[lane] = lo | (hi << 16);
        if (lane == 0) *scale = sc;
    } else {
        // scale 2^k, k = exponent - 14, at least -126 (an infinity or a NaN
        // takes the largest and stays what it is)
        const int k = max(static_cast<int>(m >> 23) - 127 - 14, -126);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        const __half2 a = __floats2half2_rn(v[0] * inv, v[1] * inv), b = __floats2half2_rn(v[2] * inv, v[3] * inv);
        reinterpret_cast<uint2*>(dst)[lane] = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                         *reinterpret_cast<const uint32_t*>(&b));
        if (lane == 0) *scale = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    }
}

// ---------------------------------------------------------------- grid barrier

struct Ctx {
    const FewParams& p;
    uint8_t* smem;
    uint64_t* full;
    uint64_t* empty;
    volatile int* abort_flag;
    int tid, warp, lane;
};

// All consumer threads of all blocks.  Writes before it are visible to reads
// (through L2) after it.
__device__ void grid_barrier(const Ctx& c, int which) {
    bar_consumers();
    if (c.tid == 0) {
        uint32_t* ctr = c.p.ctr + CTR_BAR + which;
        __threadfence();
        atomicAdd(ctr, 1u);
        if (*c.abort_flag) atomicExch(c.p.ctr + CTR_ABORT, 1u);
        const uint64_t t0 = global_timer_ns();
        for (uint32_t it = 1; !*c.abort_flag && ld_acquire(ctr) < gridDim.x; ++it) {
            if ((it & 63u) == 0) {
                if (ld_acquire(c.p.ctr + CTR_ABORT)) *c.abort_flag = 1;
                else if (global_timer_ns() - t0 > kWaitNs) {
                    *c.abort_flag = 1;
                    set_device_status(c.p.status, MOE_DEV_TIMEOUT);
                    atomicExch(c.p.ctr + CTR_ABORT, 1u);
                }
            }
        }
        __threadfence();
    }
    bar_consumers();
}

// ---------------------------------------------------------------- jobs

// A job: `rows` consecutive rows of one matrix, streamed over all of K in
// 128-byte pieces; a slot of the ring holds nk pieces (rows padded to
// 128 / nk).
struct Job {
    int shared;           // 1: shared expert
    int mat, row0, rows;
    int n, k;             // the matrix: n rows of k columns
    int nk, pieces, slots;
    uint32_t mask;        // tokens that go through it
    uint64_t kpack;       // routed: their slots
};

template <int MODE>
__device__ __forceinline__ void finish_job(Job& j, int pad_rows) {
    j.nk = pad_rows > 64 ? 1 : pad_rows > 32 ? 2 : pad_rows > 16 ? 4 : 8;
    j.pieces = (j.k + 2 * Form<MODE>::KH - 1) / (2 * Form<MODE>::KH);
    j.slots = (j.pieces + j.nk - 1) / j.nk;
}

// Phase 2: this block's share of the rows of W1, in units of 16.
template <int MODE, typename F>
__device__ __forceinline__ void for_jobs2(const Ctx& c, int n_active, F&& body) {
    const FewParams& p = c.p;
    const uint32_t* mask = reinterpret_cast<const uint32_t*>(c.smem + OFF_MASK);
    const uint64_t* kpack = reinterpret_cast<const uint64_t*>(c.smem + OFF_KPACK);
    const int* act = reinterpret_cast<const int*>(c.smem + OFF_ACT);
    const int us = p.dffs / 16, ur = p.dff / 16;
    const int n_shared = p.S * us;
    const long long units = n_shared + static_cast<long long>(n_active) * ur;
    int u = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    while (u < end) {
        Job j;
        const bool sh = u < n_shared;
        const int v = sh ? u : u - n_shared, per = sh ? us : ur;
        const int m = v / per, r = v % per;
        const int run = min(end - u, per - r);
        const int cuts = (run + 7) / 8, take = (run + cuts - 1) / cuts;
        j.shared = sh;
        j.mat = sh ? m : act[m];
        j.mask = sh ? (1u << p.T) - 1u : mask[j.mat];
        j.kpack = sh ? 0 : kpack[j.mat];
        j.row0 = 16 * r;
        j.rows = 16 * take;
        j.n = sh ? p.dffs : p.dff;
        j.k = p.d;
        finish_job<MODE>(j, j.rows);
        body(j);
        u += take;
    }
}

// Phase 3: the matrices whose products sum into one range of output rows.
template <int MODE, typename F>
__device__ __forceinline__ void for_jobs3(const Ctx& c, int n_active, int row0, int rows, F&& body) {
    const FewParams& p = c.p;
    const uint32_t* mask = reinterpret_cast<const uint32_t*>(c.smem + OFF_MASK);
    const uint64_t* kpack = reinterpret_cast<const uint64_t*>(c.smem + OFF_KPACK);
    const int* act = reinterpret_cast<const int*>(c.smem + OFF_ACT);
    for (int m = 0; m < p.S + n_active; ++m) {
        Job j;
        j.shared = m < p.S;
        j.mat = j.shared ? m : act[m - p.S];
        j.mask = j.shared ? (1u << p.T) - 1u : mask[j.mat];
        j.kpack = j.shared ? 0 : kpack[j.mat];
        j.row0 = row0;
        j.rows = rows;
        j.n = p.d;
        j.k = j.shared ? p.dffs : p.dff;
        finish_job<MODE>(j, p.rows3);
        body(j);
    }
}

// ---------------------------------------------------------------- producer

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() { if (++slot == SLOTS) { slot = 0; phase ^= 1u; } }
};

// Loads every slot of a job; false after a wait gave up.  box: rows of the
// tensor map's box (16 in phase 2; the whole job in phase 3).
template <int MODE>
__device__ __forceinline__ bool produce(const Ctx& c, const Job& j, const CUtensorMap* map, const uint8_t* scales,
                                        int box, Ring& ring, int& issued) {
    const int boxes = (j.rows + box - 1) / box;
    const int pitch = SLOT_BYTES / j.nk, srows = 128 / j.nk;
    constexpr int ELEMS = MODE == M_BF16 ? 64 : 128;        // map elements (bf16, or bytes) per piece
    const int kq = j.k / 32;
    for (int s = 0; s < j.slots; ++s) {
        uint64_t* full = c.full + ring.slot;
        const int first = s * j.nk, np = min(j.nk, j.pieces - first);
        int ok = 1;
        if (c.lane == 0) {
            ok = mbar_wait_bounded(c.empty + ring.slot, ring.phase ^ 1u, c.abort_flag, c.p.status, kWaitNs);
            if (ok) mbar_arrive_expect_tx(full, static_cast<uint32_t>(np * boxes * box * 128));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        uint8_t* dst = c.smem + OFF_RING + ring.slot * SLOT_BYTES;
        if (c.lane < np * boxes) {
            const int q = c.lane / boxes, b = c.lane % boxes;
            tma_load_3d(dst + q * pitch + b * box * 128, map, full, (first + q) * ELEMS, j.row0 + b * box, j.mat);
        }
        if (MODE == M_FP4) {
            // the 8 scale bytes of each row of each piece, as two words
            uint8_t* sdst = c.smem + OFF_SCALES + ring.slot * SCALE_BYTES;
            for (int i = c.lane; i < np * srows * 2; i += 32) {
                const int q = i / (2 * srows), r = (i >> 1) % srows, k0 = (first + q) * 8 + (i & 1) * 4;
                if (r < j.rows && j.row0 + r < j.n && k0 < kq)
                    cp_async_4(sdst + q * srows * 8 + r * 8 + (i & 1) * 4,
                               scales + (static_cast<size_t>(j.mat) * j.n + j.row0 + r) * kq + k0);
            }
            cp_async_arrive(full);
        }
        ++issued;
        ring.next();
    }
    return true;
}

// ---------------------------------------------------------------- consumer

template <int MODE, int NT>
struct BRegs {
    static constexpr int V = MODE == M_FP4 ? 4 : 1;        // 16-byte vectors per token column
    uint4 v[NT][V];
    float cs[NT][2];                                        // factors of this lane's two result columns
    float rs[2];                                            // FP8: weight scales of the job's two row blocks
};

// What the consumers need to find the token side of a job.
struct TokenSide {
    const uint8_t* base;  // operand rows
    const float* scales;  // per 128 columns, or nullptr (bf16)
    int per_slot;         // 1: row (t, slot) of routed h; 0: row t
    bool gated;           // multiply by the gate (phase 3, routed)
};

template <int MODE, int NT>
__device__ __forceinline__ void load_b(const Ctx& c, const Job& j, const TokenSide& ts, const void* wscales,
                                       int piece, BRegs<MODE, NT>& r) {
    const int g = c.lane >> 2, t4 = c.lane & 3;
    const int k0 = (2 * piece + (c.warp & 1)) * Form<MODE>::KH;
    const bool in = k0 < j.k;
    const float* gate = reinterpret_cast<const float*>(c.smem + OFF_GATE);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int t = nt * 8 + g;
        const bool on = in && (j.mask >> t & 1u);
        const int slot = static_cast<int>(j.kpack >> (4 * t)) & 15;
        const size_t row = ts.per_slot ? static_cast<size_t>(t) * c.p.K + slot : t;
        const uint8_t* src = ts.base + (row * j.k + k0) * Form<MODE>::BB;
#pragma unroll
        for (int b = 0; b < BRegs<MODE, NT>::V; ++b)
            r.v[nt][b] = on ? __ldcg(reinterpret_cast<const uint4*>(src) + 4 * b + t4) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tc = nt * 8 + 2 * t4 + i;
            const int sc = static_cast<int>(j.kpack >> (4 * tc)) & 15;
            float f = 0.f;
            if (in && (j.mask >> tc & 1u)) {
                const size_t rc = ts.per_slot ? static_cast<size_t>(tc) * c.p.K + sc : tc;
                f = MODE == M_BF16 ? 1.f : __ldcg(ts.scales + rc * (j.k / 128) + k0 / 128);
                if (ts.gated) f *= gate[tc * 16 + sc];
            }
            r.cs[nt][i] = f;
        }
    }
    if (MODE == M_FP8) {
        const float* w = static_cast<const float*>(wscales);
        const int nb = j.n / 128, kb = j.k / 128, b0 = j.row0 / 128;
        const float* q = w + (static_cast<size_t>(j.mat) * nb + b0) * kb + k0 / 128;
        r.rs[0] = in ? __ldg(q) : 0.f;
        r.rs[1] = in && b0 + 1 < nb ? __ldg(q + kb) : 0.f;
    }
}

// acc += v * cs * rs, except in the column of a token that does not go through
// the job (cs = 0): what an infinite or NaN weight makes of its zero operand
// must not reach it.
__device__ __forceinline__ void scaled_add(float& acc, float v, float cs, float rs) {
    if (cs != 0.f) acc = fmaf(v, cs * rs, acc);
}

// One piece's half (64 bytes of every row): acc += W x for the job's rows.
template <int MODE, int NT>
__device__ __forceinline__ void multiply(const Ctx& c, const Job& j, const uint8_t* piece, const uint8_t* scales,
                                         const BRegs<MODE, NT>& b, float (&acc)[8][NT][4]) {
    const int g = c.lane >> 2, t4 = c.lane & 3, half = c.warp & 1;
    const bool hi = NT == 2 && (j.mask >> 8) != 0;          // any token in the second column tile
    if (MODE == M_BF16 || MODE == M_FP8) {
        uint32_t bf[NT][8];
        if (MODE == M_FP8) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t w[4] = {b.v[nt][0].x, b.v[nt][0].y, b.v[nt][0].z, b.v[nt][0].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) e4m3x4_to_f16x2(w[q], bf[nt][2 * q], bf[nt][2 * q + 1]);
            }
        }
        const int split = (j.row0 / 128 + 1) * 128 - j.row0;   // first row of the second scale block
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            if (16 * m >= j.rows) break;
            const int r0 = 16 * m + g;
            // 16-byte chunk q of row r is at chunk q ^ (r mod 8) (128-byte swizzle); r0 and r0 + 8 swizzle alike
            const uint32_t off = static_cast<uint32_t>(r0 * 128 + (((half * 4 + t4) ^ g) << 4));
            const uint4 w0 = *reinterpret_cast<const uint4*>(piece + off);
            const uint4 w1 = *reinterpret_cast<const uint4*>(piece + off + 8 * 128);
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
            float s[NT][4] = {};
            if (MODE == M_BF16) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t bw[4] = {b.v[nt][0].x, b.v[nt][0].y, b.v[nt][0].z, b.v[nt][0].w};
                        if (nt == 0 || hi)
                            mma_bf16(s[nt], a0[2 * q], a1[2 * q], a0[2 * q + 1], a1[2 * q + 1], bw[2 * q], bw[2 * q + 1]);
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) scaled_add(acc[m][nt][i], s[nt][i], b.cs[nt][i & 1], 1.f);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t f0, f1, f2, f3;
                    e4m3x4_to_f16x2(a0[q], f0, f2);
                    e4m3x4_to_f16x2(a1[q], f1, f3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (nt == 0 || hi) mma_f16(s[nt], f0, f1, f2, f3, bf[nt][2 * q], bf[nt][2 * q + 1]);
                }
                const float rs0 = r0 < split ? b.rs[0] : b.rs[1], rs1 = r0 + 8 < split ? b.rs[0] : b.rs[1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        scaled_add(acc[m][nt][i], s[nt][i], b.cs[nt][i & 1], i < 2 ? rs0 : rs1);
            }
        }
    } else {
        // ldmatrix: matrix i holds rows 8 (i & 1) .. + 7 of block i >> 1; lane l
        // names row l & 7 of matrix l >> 3 and receives 4 bytes of row l >> 2
        const int lr = (c.lane & 7) + ((c.lane >> 3) & 1) * 8, lb = c.lane >> 4;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            if (16 * m >= j.rows) break;
            const uint32_t s0 = *reinterpret_cast<const uint32_t*>(scales + (16 * m + g) * 8 + half * 4);
            const uint32_t s1 = *reinterpret_cast<const uint32_t*>(scales + (16 * m + g + 8) * 8 + half * 4);
            float s[NT][4] = {};
#pragma unroll
            for (int pr = 0; pr < 2; ++pr) {                 // two pairs of blocks
                const int chunk = half * 4 + pr * 2 + lb;
                const uint32_t addr = smem_u32(piece) + static_cast<uint32_t>((16 * m + lr) * 128 + ((chunk ^ (lr & 7)) << 4));
                uint32_t w[4];
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
#pragma unroll
                for (int bb = 0; bb < 2; ++bb) {
                    const int blk = pr * 2 + bb;
                    uint32_t a0[4], a1[4];
                    e2m1x8_to_f16x2(w[2 * bb], a0);
                    e2m1x8_to_f16x2(w[2 * bb + 1], a1);
                    const float rs0 = e8m0_value((s0 >> (8 * blk)) & 255u), rs1 = e8m0_value((s1 >> (8 * blk)) & 255u);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (nt && !hi) continue;
                        const uint4 bv = b.v[nt][blk];
                        float t[4] = {};
                        mma_f16(t, a0[0], a1[0], a0[1], a1[1], bv.x, bv.y);
                        mma_f16(t, a0[2], a1[2], a0[3], a1[3], bv.z, bv.w);
                        s[nt][0] = fmaf(t[0], rs0, s[nt][0]);
                        s[nt][1] = fmaf(t[1], rs0, s[nt][1]);
                        s[nt][2] = fmaf(t[2], rs1, s[nt][2]);
                        s[nt][3] = fmaf(t[3], rs1, s[nt][3]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) scaled_add(acc[m][nt][i], s[nt][i], b.cs[nt][i & 1], 1.f);
        }
    }
}

// Streams a job's slots.  Warp w takes the pieces congruent to w / 2 modulo 4
// and of each the half w & 1; every slot's empty barrier counts 8 arrivals
// from the warps that have a piece in it.
template <int MODE, int NT>
__device__ __forceinline__ void consume(const Ctx& c, const Job& j, const TokenSide& ts, const void* wscales,
                                        Ring& ring, bool& ok, float (&acc)[8][NT][4]) {
    const int mine = c.warp >> 1;
    const int pitch = SLOT_BYTES / j.nk, spitch = SCALE_BYTES / j.nk;
    const uint32_t weight = j.nk == 1 ? 4u : j.nk == 2 ? 2u : 1u;
    BRegs<MODE, NT> cur, nxt;
    if (mine < j.pieces) load_b<MODE, NT>(c, j, ts, wscales, mine, cur);
    for (int s = 0; s < j.slots; ++s, ring.next()) {
        const int first = s * j.nk;
        if (j.nk == 1 && (s & 3) != mine) continue;
        if (j.nk == 2 && (s & 1) != mine >> 1) continue;
        const int q0 = j.nk == 1 ? 0 : j.nk == 2 ? (mine & 1) : mine;
        if (ok) {
            int w = 1;
            if (c.lane == 0) w = mbar_wait_bounded(c.full + ring.slot, ring.phase, c.abort_flag, c.p.status, kWaitNs);
            ok = __shfl_sync(0xffffffffu, w, 0) != 0;
        }
        for (int q = q0; q < j.nk; q += 4) {
            const int piece = first + q;
            if (piece >= j.pieces) break;
            if (piece + 4 < j.pieces) load_b<MODE, NT>(c, j, ts, wscales, piece + 4, nxt);
            if (ok && (2 * piece + (c.warp & 1)) * Form<MODE>::KH < j.k)
                multiply<MODE, NT>(c, j, c.smem + OFF_RING + ring.slot * SLOT_BYTES + q * pitch,
                                   c.smem + OFF_SCALES + ring.slot * SCALE_BYTES + q * spitch, cur, acc);
            cur = nxt;
        }
        __syncwarp();
        if (c.lane == 0) mbar_arrive_n(c.empty + ring.slot, weight);
    }
}

// The sum over the warps of one column tile's accumulators, in warp order:
// body(row, column of the tile, sum) for every row below `rows`.  Every
// consumer thread calls it; the buffer is free again afterwards.
template <int NT, typename F>
__device__ __forceinline__ void reduce_tile(const Ctx& c, int nt, int rows, const float (&acc)[8][NT][4], F&& body) {
    float* red = reinterpret_cast<float*>(c.smem + OFF_RED);
    const int g = c.lane >> 2, t4 = c.lane & 3;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        if (16 * m >= rows) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = acc[m][0][i];
            if (NT == 2 && nt == 1) v = acc[m][NT - 1][i];
            red[(c.warp * 8 + 2 * t4 + (i & 1)) * RED_PITCH + 16 * m + g + 8 * (i >> 1)] = v;
        }
    }
    bar_consumers();
    for (int i = c.tid; i < rows * 8; i += CT) {
        const int col = i / rows, r = i % rows;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < CW; ++w) v += red[(w * 8 + col) * RED_PITCH + r];
        body(r, col, v);
    }
    bar_consumers();
}

// ---------------------------------------------------------------- phase 1

template <int MODE, int NT>
__device__ __forceinline__ void router_and_x(const Ctx& c) {
    const FewParams& p = c.p;
    if (MODE != M_BF16) {
        const int nb = p.d / 128;
        for (int i = blockIdx.x * CW + c.warp; i < p.T * nb; i += gridDim.x * CW) {
            const int t = i / nb, b = i % nb;
            const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.d + b * 128) + c.lane);
            const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                                __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
            store_block<MODE>(v, p.xq + (static_cast<size_t>(t) * p.d + b * 128) * Form<MODE>::BB,
                              p.xs + static_cast<size_t>(t) * nb + b, c.lane);
        }
    }
    // items (slice, expert), slice-major: a block mostly stays in one slice of
    // x, which it stages in the ring's memory
    const int items = p.ks * p.E;
    int i0 = static_cast<int>(static_cast<long long>(items) * blockIdx.x / gridDim.x);
    const int i1 = static_cast<int>(static_cast<long long>(items) * (blockIdx.x + 1) / gridDim.x);
    __nv_bfloat16* xsm = reinterpret_cast<__nv_bfloat16*>(c.smem + OFF_RING);
    while (i0 < i1) {
        const int ks = i0 / p.E, e0 = i0 % p.E, e1 = min(p.E, e0 + i1 - i0);
        const int k0 = ks * p.slice, len = min(p.slice, p.d - k0);       // multiples of 64
        bar_consumers();
        for (int i = c.tid; i < p.T * (len / 8); i += CT) {
            const int t = i / (len / 8), q = i % (len / 8);
            reinterpret_cast<uint4*>(xsm + t * p.slice)[q] =
                __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.d + k0) + q);
        }
        bar_consumers();
        for (int e = e0 + c.warp; e < e1; e += CW) {
            const float4* w = reinterpret_cast<const float4*>(p.W_r + static_cast<size_t>(e) * p.d + k0);
            float acc[8 * NT] = {};
#pragma unroll 4
            for (int q = c.lane; q < len / 4; q += 32) {
                const float4 wv = __ldg(w + q);
#pragma unroll
                for (int t = 0; t < 8 * NT; ++t) {
                    if (t < p.T) {
                        const uint2 xv = *reinterpret_cast<const uint2*>(xsm + t * p.slice + 4 * q);
                        acc[t] = fmaf(__uint_as_float(xv.x << 16), wv.x, acc[t]);
                        acc[t] = fmaf(__uint_as_float(xv.x & 0xFFFF0000u), wv.y, acc[t]);
                        acc[t] = fmaf(__uint_as_float(xv.y << 16), wv.z, acc[t]);
                        acc[t] = fmaf(__uint_as_float(xv.y & 0xFFFF0000u), wv.w, acc[t]);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 8 * NT; ++t) {
                if (t >= p.T) break;
                float v = acc[t];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (c.lane == t) p.part[(static_cast<size_t>(ks) * p.T + t) * p.E + e] = v;
            }
        }
        i0 += e1 - e0;
    }
}

// ---------------------------------------------------------------- selection

// Order-preserving key of a float, at least 1 (0 marks a taken expert).
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return max(b & 0x80000000u ? ~b : b | 0x80000000u, 1u);
}

// Top-K, gates and the list of experts reached, by every block for itself;
// the last block also writes the routing outputs and the balance statistics.
// Returns the number of experts reached (the same in every thread).
__device__ int select_experts(const Ctx& c) {
    const FewParams& p = c.p;
    int* idx_s = reinterpret_cast<int*>(c.smem + OFF_IDX);
    float* gate_s = reinterpret_cast<float*>(c.smem + OFF_GATE);
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(c.smem + OFF_MASK);
    uint64_t* kpack_s = reinterpret_cast<uint64_t*>(c.smem + OFF_KPACK);
    int* act_s = reinterpret_cast<int*>(c.smem + OFF_ACT);
    int* misc = reinterpret_cast<int*>(c.smem + OFF_MISC);
    float* prob_s = reinterpret_cast<float*>(c.smem + OFF_RED);       // [T][256], last block only
    const bool writer = blockIdx.x == gridDim.x - 1;
    for (int t = c.warp; t < p.T; t += CW) {
        float l[8];
        uint32_t key[8];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 32 * i + c.lane;
            l[i] = -INFINITY;
            key[i] = 0;
            if (e < p.E) {
                float v = 0.f;
#pragma unroll 4
                for (int s = 0; s < p.ks; ++s) v += __ldcg(p.part + (static_cast<size_t>(s) * p.T + t) * p.E + e);
                if (p.logit_bias) v += __ldg(p.logit_bias + e);
                l[i] = v;
                key[i] = order_key(p.sel_bias ? v + __ldg(p.sel_bias + e) : v);
                top = fmaxf(top, v);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[i] = expf(l[i] - top);
            sum += l[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (writer) {
#pragma unroll
            for (int i = 0; i < 8; ++i) prob_s[t * 256 + 32 * i + c.lane] = l[i] / sum;
        }
        float chosen = 0.f, mine = 0.f;
        for (int k = 0; k < p.K; ++k) {
            uint32_t bk = 0, bi = 0xFFFFu;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (key[i] > bk) { bk = key[i]; bi = 32 * i + c.lane; }
            const uint32_t best = __reduce_max_sync(0xffffffffu, bk);
            const uint32_t e = __reduce_min_sync(0xffffffffu, bk == best ? bi : 0xFFFFu);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e == static_cast<uint32_t>(32 * i + c.lane)) { v = l[i]; key[i] = 0; }
            v = __shfl_sync(0xffffffffu, v, e & 31);
            chosen += v;
            if (c.lane == k) mine = v;
            if (c.lane == 0) idx_s[t * 16 + k] = static_cast<int>(e);
        }
        if (c.lane < p.K) gate_s[t * 16 + c.lane] = mine / chosen;
    }
    bar_consumers();
    // one thread per expert: its slots in capacity order
    const int e = c.tid;
    int count = 0, kept = 0;
    uint32_t mask = 0;
    uint64_t kpack = 0;
    const int cap = p.capacity < 0 ? MAX_T : p.capacity;
    auto slot = [&](int t, int k) {
        if (idx_s[t * 16 + k] == e) {
            ++count;
            if (kept < cap) {
                ++kept;
                mask |= 1u << t;
                kpack |= static_cast<uint64_t>(k) << (4 * t);
            }
        }
    };
    if (p.slot_major) {
        for (int k = 0; k < p.K; ++k)
            for (int t = 0; t < p.T; ++t) slot(t, k);
    } else {
        for (int t = 0; t < p.T; ++t)
            for (int k = 0; k < p.K; ++k) slot(t, k);
    }
    mask_s[e] = mask;
    kpack_s[e] = kpack;
    const uint32_t votes = __ballot_sync(0xffffffffu, mask != 0);
    if (c.lane == 0) misc[4 + c.warp] = __popc(votes);
    bar_consumers();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
        const int n = misc[4 + w];
        if (w < c.warp) base += n;
        total += n;
    }
    if (mask) act_s[base + __popc(votes & ((1u << c.lane) - 1u))] = e;
    if (c.tid == 0) misc[1] = total;
    if (writer) {
        for (int i = c.tid; i < p.T * p.K; i += CT) {
            if (p.topk_idx) p.topk_idx[i] = idx_s[(i / p.K) * 16 + i % p.K];
            if (p.gates) p.gates[i] = gate_s[(i / p.K) * 16 + i % p.K];
        }
        float* prod = prob_s + MAX_T * 256;
        float fp = 0.f;
        if (e < p.E) {
            float P = 0.f;
            for (int t = 0; t < p.T; ++t) P += prob_s[t * 256 + e];
            P /= p.T;
            const float f = static_cast<float>(count) / static_cast<float>(p.T * p.K);
            p.P[e] = P;
            p.f[e] = f;
            if (p.counts) p.counts[e] = count;
            fp = f * P;
        }
        prod[e] = fp;
        bar_consumers();
        if (c.warp == 0) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += prod[8 * c.lane + i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (c.lane == 0) *p.loss = p.alpha * p.E * v;
        }
        bar_consumers();
    }
    return total;
}

// ---------------------------------------------------------------- the kernel

template <int MODE, int NT>
__global__ void __launch_bounds__(THREADS, 1)
few_tokens_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    int* misc = reinterpret_cast<int*>(smem + OFF_MISC);
    const Ctx c{p, smem, full, full + SLOTS, misc, static_cast<int>(threadIdx.x), static_cast<int>(threadIdx.x >> 5),
                static_cast<int>(threadIdx.x & 31)};
    if (c.tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(c.full + i, MODE == M_FP4 ? 33 : 1);      // expect_tx, and a lane each of the scale copies
            mbar_init(c.empty + i, CW);
        }
        misc[0] = 0;
        fence_mbar_init();
    }
    __syncthreads();

    const int row_begin = static_cast<int>(static_cast<long long>(p.d) * blockIdx.x / gridDim.x);
    const int row_end = static_cast<int>(static_cast<long long>(p.d) * (blockIdx.x + 1) / gridDim.x);

    if (c.warp == CW) {
        // ================= producer
        if (c.lane == 0) {
            tma_prefetch_desc(&p.w1);
            tma_prefetch_desc(&p.w2);
            if (p.S) { tma_prefetch_desc(&p.ws1); tma_prefetch_desc(&p.ws2); }
        }
        __syncthreads();                                        // the experts are selected
        const int n_active = misc[1];
        Ring ring;
        int issued = 0;
        bool ok = *c.abort_flag == 0;
        for_jobs2<MODE>(c, n_active, [&](const Job& j) {
            if (ok) ok = produce<MODE>(c, j, j.shared ? &p.ws1 : &p.w1,
                                       static_cast<const uint8_t*>(j.shared ? p.ws1s : p.w1s), 16, ring, issued);
        });
        for (int r = row_begin; r < row_end; r += p.rows3)
            for_jobs3<MODE>(c, n_active, r, min(p.rows3, row_end - r), [&](const Job& j) {
                if (ok) ok = produce<MODE>(c, j, j.shared ? &p.ws2 : &p.w2,
                                           static_cast<const uint8_t*>(j.shared ? p.ws2s : p.w2s), p.rows3, ring, issued);
            });
        if (MODE == M_FP4) asm volatile("cp.async.wait_all;" ::: "memory");
        // copies in flight land before the block gives its memory back
        if (c.lane == 0) {
            int s = ring.slot;
            uint32_t ph = ring.phase;
            for (int i = 0; i < min(issued, SLOTS); ++i) {
                if (--s < 0) { s = SLOTS - 1; ph ^= 1u; }
                volatile int no_abort = 0;
                mbar_wait_bounded(c.full + s, ph, &no_abort, nullptr, kDrainNs);
            }
        }
        __syncwarp();
    } else {
        // ================= consumers
        router_and_x<MODE, NT>(c);
        grid_barrier(c, 0);
        const int n_active = select_experts(c);
        fence_proxy_async_smem();       // phase 1 used the ring's memory
        __syncthreads();
        Ring ring;
        bool ok = *c.abort_flag == 0;
        float acc[8][NT][4];
        const size_t h_shared = static_cast<size_t>(p.T) * p.K * p.dff;   // first element of the shared rows of h
        for_jobs2<MODE>(c, n_active, [&](const Job& j) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;
            const TokenSide ts{p.xq, p.xs, 0, false};
            consume<MODE, NT>(c, j, ts, j.shared ? p.ws1s : p.w1s, ring, ok, acc);
            const float* bias = (j.shared ? p.bs1 : p.b1) + static_cast<size_t>(j.mat) * j.n + j.row0;
            const size_t base = j.shared ? h_shared + static_cast<size_t>(j.mat) * p.T * j.n : 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt && !(j.mask >> 8)) continue;
                reduce_tile<NT>(c, nt, j.rows, acc, [&](int r, int col, float v) {
                    const int t = nt * 8 + col;
                    if (!(j.mask >> t & 1u)) return;
                    const int slot = static_cast<int>(j.kpack >> (4 * t)) & 15;
                    const size_t row = j.shared ? t : static_cast<size_t>(t) * p.K + slot;
                    const float h = silu_fast(v + __ldg(bias + r));
                    const size_t at = base + row * j.n + j.row0 + r;
                    if (MODE == M_BF16) reinterpret_cast<__nv_bfloat16*>(p.hq)[at] = __float2bfloat16_rn(h);
                    else p.h32[at] = h;
                });
            }
        });
        grid_barrier(c, 1);
        const size_t hs_shared = h_shared / 128;
        if (MODE != M_BF16) {
            // a warp per 128 values of h that phase 3 reads
            const int* idx_s = reinterpret_cast<const int*>(smem + OFF_IDX);
            const uint32_t* mask_s = reinterpret_cast<const uint32_t*>(smem + OFF_MASK);
            const uint64_t* kpack_s = reinterpret_cast<const uint64_t*>(smem + OFF_KPACK);
            const int nr = p.dff / 128, ns = p.dffs / 128;
            const int routed = p.T * p.K * nr, all = routed + p.S * p.T * ns;
            for (int i = blockIdx.x * CW + c.warp; i < all; i += gridDim.x * CW) {
                size_t blk;
                if (i < routed) {
                    const int s = i / nr, t = s / p.K, k = s % p.K, e = idx_s[t * 16 + k];
                    // a slot over the capacity has no h
                    if (!(mask_s[e] >> t & 1u) || (static_cast<int>(kpack_s[e] >> (4 * t)) & 15) != k) continue;
                    blk = i;
                } else {
                    blk = hs_shared + (i - routed);
                }
                const float4 q = __ldcg(reinterpret_cast<const float4*>(p.h32 + blk * 128) + c.lane);
                const float v[4] = {q.x, q.y, q.z, q.w};
                store_block<MODE>(v, p.hq + blk * 128 * Form<MODE>::BB, p.hs + blk, c.lane);
            }
            grid_barrier(c, 2);
        }
        const int* idx_s = reinterpret_cast<const int*>(smem + OFF_IDX);
        const float* gate_s = reinterpret_cast<const float*>(smem + OFF_GATE);
        const uint32_t* mask_s = reinterpret_cast<const uint32_t*>(smem + OFF_MASK);
        for (int r0 = row_begin; r0 < row_end; r0 += p.rows3) {
            const int rows = min(p.rows3, row_end - r0);
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;
            for_jobs3<MODE>(c, n_active, r0, rows, [&](const Job& j) {
                const size_t at = j.shared ? h_shared + static_cast<size_t>(j.mat) * p.T * j.k : 0;
                const TokenSide ts{p.hq + at * Form<MODE>::BB, p.hs + at / 128, !j.shared, !j.shared};
                consume<MODE, NT>(c, j, ts, j.shared ? p.ws2s : p.w2s, ring, ok, acc);
            });
            ok = ok && *c.abort_flag == 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                reduce_tile<NT>(c, nt, rows, acc, [&](int r, int col, float v) {
                    const int t = nt * 8 + col;
                    if (t >= p.T || !ok) return;
                    const int row = r0 + r;
                    for (int k = 0; k < p.K; ++k) {
                        const int e = idx_s[t * 16 + k];
                        const float g = gate_s[t * 16 + k];
                        if (mask_s[e] >> t & 1u) v = fmaf(g, __ldg(p.b2 + static_cast<size_t>(e) * p.d + row), v);
                        else if (p.passthrough)
                            v = fmaf(g, __bfloat162float(p.x[static_cast<size_t>(t) * p.d + row]), v);
                    }
                    for (int s = 0; s < p.S; ++s) v += __ldg(p.bs2 + static_cast<size_t>(s) * p.d + row);
                    p.out[static_cast<size_t>(t) * p.d + row] = __float2bfloat16_rn(v);
                });
            }
        }
    }
    __syncthreads();
    // the last block to leave zeroes the counters for the next launch
    if (c.tid == 0) {
        __threadfence();
        if (atomicAdd(p.ctr + CTR_EXIT, 1u) == gridDim.x - 1) {
            for (int i = 0; i < CTR_WORDS; ++i) p.ctr[i] = 0;
            __threadfence();
        }
    }
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct FewLayout {
    size_t ctr, part, xq, xs, h32, hq, hs, total;
};

// blocks: as many as can find work, at most one per SM
struct FewPlan {
    int blocks, ks, slice;
};

FewPlan few_plan(const Dims& dm, int sms) {
    FewPlan f;
    // a warp per (expert, slice); slices are multiples of 128 columns, at most
    // 5120 of them (16 tokens' slice of x fills the ring's memory)
    static_assert(MAX_T * 5120 * 2 <= SLOTS * SLOT_BYTES, "the staged slice of x fits the ring");
    const int want = (sms * CW + dm.E - 1) / dm.E;
    const int pieces = (dm.d + 127) / 128;
    int per = (pieces + want - 1) / want;
    if (per > 40) per = 40;
    f.slice = 128 * per;
    f.ks = (pieces + per - 1) / per;
    const long long units = (static_cast<long long>(dm.T) * dm.K * dm.dff + static_cast<long long>(dm.S) * dm.dffs) / 16;
    long long b = units;
    if (b < dm.d / 16) b = dm.d / 16;
    if (b < (f.ks * dm.E + CW - 1) / CW) b = (f.ks * dm.E + CW - 1) / CW;
    f.blocks = b < sms ? static_cast<int>(b < 1 ? 1 : b) : sms;
    return f;
}

FewLayout few_layout(const Dims& dm) {
    FewLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off = align256(off + bytes); return o; };
    const bool q = dm.dtype != MOE_BF16;
    const size_t bb = dm.dtype == MOE_FP8_E4M3_BLOCK ? 1 : 2;
    const size_t h = static_cast<size_t>(dm.T) * dm.K * dm.dff + static_cast<size_t>(dm.S) * dm.T * dm.dffs;
    take(256);                                              // status word
    L.ctr = take(256);
    // slices are at least 128 columns long, whatever the device's size
    L.part = take(static_cast<size_t>((dm.d + 127) / 128) * dm.T * dm.E * 4);
    L.xq = take(q ? static_cast<size_t>(dm.T) * dm.d * bb : 0);
    L.xs = take(q ? static_cast<size_t>(dm.T) * (dm.d / 128) * 4 : 0);
    L.h32 = take(q ? h * 4 : 0);
    L.hq = take(h * bb);
    L.hs = take(q ? h / 128 * 4 : 0);
    L.total = off;
    return L;
}

template <int MODE, int NT>
cudaError_t launch_mode(const FewParams& p, int blocks, cudaStream_t st) {
    auto kernel = few_tokens_kernel<MODE, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_ALLOC;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t few_ws_bytes(const Dims& dm) { return few_layout(dm).total; }

cudaError_t launch_few(const Dims& dm, const FewArgs& a, void* ws, cudaStream_t st) {
    FewParams p;
    std::memset(&p, 0, sizeof(p));
    const FewLayout L = few_layout(dm);
    uint8_t* w = static_cast<uint8_t*>(ws);
    const FewPlan plan = few_plan(dm, device_sm_count());
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.W_r = a.W_r;
    p.logit_bias = dm.bias_mode == MOE_BIAS_LOGITS ? a.logit_bias : nullptr;
    p.sel_bias = dm.bias_mode == MOE_BIAS_SELECTION ? a.logit_bias : nullptr;
    p.w1s = a.W1_scales;
    p.w2s = a.W2_scales;
    p.ws1s = a.Ws1_scales;
    p.ws2s = a.Ws2_scales;
    p.b1 = a.b1;
    p.b2 = a.b2;
    p.bs1 = a.bs1;
    p.bs2 = a.bs2;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.f = a.f;
    p.P = a.P;
    p.loss = a.loss;
    p.topk_idx = a.topk_idx;
    p.gates = a.gates;
    p.counts = a.counts;
    p.status = reinterpret_cast<int32_t*>(w);
    p.ctr = reinterpret_cast<uint32_t*>(w + L.ctr);
    p.part = reinterpret_cast<float*>(w + L.part);
    p.xq = dm.dtype == MOE_BF16 ? const_cast<uint8_t*>(static_cast<const uint8_t*>(a.x)) : w + L.xq;
    p.xs = reinterpret_cast<float*>(w + L.xs);
    p.h32 = reinterpret_cast<float*>(w + L.h32);
    p.hq = w + L.hq;
    p.hs = reinterpret_cast<float*>(w + L.hs);
    p.alpha = dm.alpha;
    p.T = dm.T;
    p.d = dm.d;
    p.E = dm.E;
    p.K = dm.K;
    p.dff = dm.dff;
    p.S = dm.S;
    p.dffs = dm.dffs;
    p.capacity = dm.capacity;
    p.slot_major = dm.slot_major;
    p.passthrough = dm.passthrough;
    p.ks = plan.ks;
    p.slice = plan.slice;
    const int most = (dm.d + plan.blocks - 1) / plan.blocks;
    p.rows3 = most < 128 ? most : 128;
    const int elem = dm.dtype == MOE_BF16 ? 2 : 1;
    const int div = dm.dtype == MOE_MXFP4 ? 2 : 1;           // elements of K per map element
    if (!encode_tma_3d(&p.w1, a.W1, dm.E, dm.dff, dm.d / div, elem, 16) ||
        !encode_tma_3d(&p.w2, a.W2, dm.E, dm.d, dm.dff / div, elem, p.rows3))
        return cudaErrorInvalidValue;
    if (dm.S > 0 && (!encode_tma_3d(&p.ws1, a.Ws1, dm.S, dm.dffs, dm.d / div, elem, 16) ||
                     !encode_tma_3d(&p.ws2, a.Ws2, dm.S, dm.d, dm.dffs / div, elem, p.rows3)))
        return cudaErrorInvalidValue;
    const bool two = dm.T > 8;
    if (dm.dtype == MOE_BF16)
        return two ? launch_mode<M_BF16, 2>(p, plan.blocks, st) : launch_mode<M_BF16, 1>(p, plan.blocks, st);
    if (dm.dtype == MOE_FP8_E4M3_BLOCK)
        return two ? launch_mode<M_FP8, 2>(p, plan.blocks, st) : launch_mode<M_FP8, 1>(p, plan.blocks, st);
    return two ? launch_mode<M_FP4, 2>(p, plan.blocks, st) : launch_mode<M_FP4, 1>(p, plan.blocks, st);
}

}  // namespace moe
