// Grouped product of MXFP4 operands on tcgen05: y[r] = act(W_e a[r] + b_e)
// for the rows r of each segment and the segment's matrix e.
//
// tcgen05.mma kind::mxf4.block_scale.scale_vec::2X multiplies packed E2M1
// operands, 64 elements of K per instruction, and applies one E8M0 scale per
// row (of A) and column (of B) per 32 elements from tensor memory; the
// accumulator sums sa * sb * (a . b) over the whole K loop in fp32.
//
// Tiles are 128 rows x 256 weight rows, one persistent CTA per SM, the
// segment table and tile order of ffn_common.cuh.  The two accumulators
// overlap in tensor memory (columns 0..255 and 192..447) and the scales take
// columns 448..495: two slots of 24, used in turn by the K stages.  The
// epilogue drains the 64 overlapping columns first.
//
// Per CTA (480 threads):
//   warp 0      TMA producer: 128 bytes of K (256 elements) per stage, A 16 KB
//               and B 32 KB;
//   warp 1      MMA issuer: per stage copies the scales from shared to tensor
//               memory (tcgen05.cp 32x128b.warpx4, in order with the MMAs),
//               then 4 MMAs of K = 64.  The warp runs the loop as a whole and
//               one elected lane issues, so that descriptors are warp-uniform
//               (a loop that one lane runs alone took 2600 cycles a stage);
//   warps 2..9  epilogue, two warps per quadrant of tensor memory (with one the
//               epilogue was busy 95 % of the time): bias, SiLU, and bf16, fp32
//               or MXFP4 rows (a chunk of 32 columns is one block of the
//               output), stored a 32-byte sector of its row per lane;
//   warps 10..13 scale loaders: a thread reads the scale bytes of its A row and
//               of two weight rows, 8 of each per stage, four stages at once
//               where K allows (one stage at once: 331 us instead of 319 for
//               8191 x 14336 x 4096), and lays them out in shared memory as tcgen05.cp reads them:
//               512 bytes per 128 rows and 128 elements of K, row r's four
//               bytes at 16 (r mod 32) + 4 (r div 32).  Their scattered reads
//               are later than the TMA's: with a ring twice as long as the
//               codes' they run ahead of them (4096-token experts 1041 -> 952 us
//               in runs of their own);
//   warp 14     relay: makes the proxy fence for a slot of scales, which in a
//               loader would wait for the reads it has in flight.
// Measured: 8191 rows x 14336 x 4096 in 273 us alone, 3.5 PFLOP/s (its MMAs
// in flight 43 % of the cycles), 379 in a row of launches at the power limit;
// 1024 rows of 256 experts, both layers, 392 to 436 us, 6.2 to 5.6 TB/s of
// weights; 32768 rows, 952 us in a run of its own and 1055 to 1142 in a row of
// launches, at the power limit.  CTA pairs (256 x 256 tiles) were 1.2 to 1.5
// times slower.
// Every wait is bounded (common.cuh).
#include "ffn_common.cuh"
#include "mxfp4.cuh"

namespace moe {
namespace {

using namespace ffn;

constexpr int EPI_WARPS = 8, LOADERS = 2 + EPI_WARPS, RELAY = LOADERS + 4, NUM_THREADS = 32 * (RELAY + 1);
constexpr int BN = 256, BKB = 128;                   // weight rows per tile; bytes of K per stage (256 elements)
constexpr uint32_t TMEM_COLS = 512, ACC1_COL = 192, SF_COL0 = 448, SF_STRIDE = 24;
constexpr int LOOKAHEAD = 4;                         // stages of scales a loader has in flight in registers
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;
constexpr uint64_t kDrainTimeoutNs = 200000000ull;

constexpr int STAGES = 4, SF_STAGES = 2 * STAGES;     // scales run ahead of the codes
constexpr int FEW_ROWS = 16;                         // rows of the short box of A
constexpr int A_BYTES = BM * BKB, B_BYTES = BN * BKB;
constexpr int SF_BYTES = 2 * 3 * 512;                // per half stage: A, B rows 0..127, B rows 128..255
constexpr int OFF_A = 0;
constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
constexpr int OFF_SF = OFF_B + STAGES * B_BYTES;
constexpr int OFF_BAR = OFF_SF + SF_STAGES * SF_BYTES;
constexpr int N_BARS = STAGES + 3 * SF_STAGES + 4 + 2;   // full; empty, sfull, sready; accf, acce [2]; ovl; drain
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int OFF_SEG = OFF_MISC + 16;
constexpr int OFF_BIAS = (OFF_SEG + SegTable::SEG_INTS * 4 + 15) & ~15;   // 2 x BN fp32, the tiles in flight
constexpr int TOTAL = OFF_BIAS + 2 * BN * 4;
constexpr int ALLOC = TOTAL + 1024;
static_assert(ALLOC <= 227 * 1024, "shared memory budget");
static_assert(OFF_SF % 128 == 0 && OFF_BAR % 8 == 0, "alignment");
static_assert(SF_COL0 + 2 * SF_STRIDE <= TMEM_COLS, "tensor memory budget");

struct __align__(64) Mx4Params {
    TcParams tc;              // a_map[0], b_map[0] over bytes; g[0].K, N in elements
    const uint8_t* a_scales;  // (rows, K/32)
    const uint8_t* w_scales;  // (n_mats, N, K/32)
    uint8_t* y_scales;        // (rows, N/32), MXFP4 output
    CUtensorMap rest_map;     // the rows of A's stage below the short box
    int wide_rows;            // y's rows start on 32-byte boundaries
    int wide_scales;          // the scales' rows do
};

// The MMA thread's wait for a full stage: bounded, polling without the
// suspend hint (this thread is on the critical path).
static __device__ __noinline__ bool mma_wait_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                  int32_t* status, uint64_t timeout_ns) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > timeout_ns) {
                *abort_flag = 1;
                set_device_status(status, MOE_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

struct Item {
    int tile, kb;
    TileInfo ti;
};

// OUT: MOE_F32, MOE_BF16 or MOE_MXFP4 rows.
template <int OUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
mxfp4_matmul_kernel(const __grid_constant__ Mx4Params mp) {
    const TcParams& p = mp.tc;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* sfull = empty + SF_STAGES;
    uint64_t* sready = sfull + SF_STAGES;
    uint64_t* accf = sready + SF_STAGES;
    uint64_t* acce = accf + 2;
    uint64_t* ovl = acce + 2;
    uint64_t* drain = ovl + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    SegTable seg(reinterpret_cast<int*>(smem + OFF_SEG));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 0) tmem_alloc<TMEM_COLS>(tmem_slot);
    if (warp == 1 && lane == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
        for (int i = 0; i < SF_STAGES; ++i) { mbar_init(&empty[i], 1); mbar_init(&sfull[i], 4); mbar_init(&sready[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&accf[i], 1); mbar_init(&acce[i], EPI_WARPS); }
        mbar_init(ovl, EPI_WARPS);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) { tma_prefetch_desc(&p.a_map[0]); tma_prefetch_desc(&p.a_map[1]); tma_prefetch_desc(&mp.rest_map); tma_prefetch_desc(&p.b_map[0]); }
    // zeros in A's stages, of which short tiles load only a part
    for (int i = tid; i < STAGES * A_BYTES / 16; i += NUM_THREADS)
        reinterpret_cast<uint4*>(smem + OFF_A)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    pdl_wait();
    pdl_allow_next();
    const int nseg = build_seg_table<BN>(p, seg, NUM_THREADS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total_tiles = seg.start[nseg];
    const int K = p.g[0].K, N = p.g[0].N;
    const int kblocks = ceil_div(K, 2 * BKB);

    // Item i (a K stage of a tile, counted over the CTA's tiles) has its codes
    // in stage i mod STAGES and its scales in slot i mod SF_STAGES; empty[slot]
    // reports its MMAs done.
    if (warp == 0) {
        // ================= TMA producer
        if (lane == 0) {
            int stage = 0, issued = 0, slot = SF_STAGES - STAGES;        // slot: of the item STAGES before
            uint32_t phase = 0, eph = 1, dirty = 0;                      // dirty: stages with rows below the short box
            bool ok = true;
            for (int tile = blockIdx.x; tile < total_tiles && ok; tile += gridDim.x) {
                const TileInfo ti = decode_tile<BN, 2 * BKB>(tile, p, seg, nseg);
                // Few rows left: the short box has them, and the rows below it
                // are zeros (left so by a short tile before, or a box that
                // lies past A's end).  Nothing reads their results, but long
                // runs of experts are at the power limit, and zeros take less
                // of it (1024 rows of 256 experts: 504 -> 462 us, 32768 rows: 1205 -> 1195).
                const int few = ti.rows_left <= FEW_ROWS;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&empty[slot], eph, abort_flag, p.status, p.timeout_ns)) { ok = false; break; }
                    if (++slot == SF_STAGES) { slot = 0; eph ^= 1u; }
                    const bool clear = few && (dirty >> stage & 1u);
                    dirty = few ? dirty & ~(1u << stage) : dirty | 1u << stage;
                    mbar_arrive_expect_tx(&full[stage], (few && !clear ? FEW_ROWS * BKB : A_BYTES) + B_BYTES);
                    if (clear)
                        tma_load_2d(smem + OFF_A + stage * A_BYTES + FEW_ROWS * BKB, &mp.rest_map, &full[stage], 0, p.g[0].a_rows);
                    tma_load_2d(smem + OFF_A + stage * A_BYTES, &p.a_map[few], &full[stage], kb * BKB, ti.a_row);
                    tma_load_3d(smem + OFF_B + stage * B_BYTES, &p.b_map[0], &full[stage], kb * BKB, ti.n0, ti.mat);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) {
                // copies in flight land before the CTA gives its memory back
                int s = stage;
                uint32_t ph = phase;
                const int pending = issued < STAGES ? issued : STAGES;
                for (int i = 0; i < pending; ++i) {
                    if (--s < 0) { s = STAGES - 1; ph ^= 1u; }
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&full[s], ph, &no_abort, nullptr, kDrainTimeoutNs);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer
        const bool leader = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
            return __all_sync(0xffffffffu, mma_wait_spin(bar, parity, abort_flag, p.status, p.timeout_ns)) != 0;
        };
        int stage = 0, sslot = 0, abuf = 0, item = 0;
        uint32_t phase = 0, sph = 0, aph0 = 0, aph1 = 0, ovl_ph = 0;
        bool ok = true, first = true;
#pragma unroll 1
        for (int tile = blockIdx.x; tile < total_tiles && ok; tile += gridDim.x) {
            // the previous tile's overlapping columns drained, and this
            // buffer's tile from two tiles back fully drained
            if (!first) {
                if (!wait(ovl, ovl_ph)) { ok = false; break; }
                ovl_ph ^= 1u;
            }
            first = false;
            uint32_t& aph = abuf ? aph1 : aph0;
            if (!wait(&acce[abuf], aph ^ 1u)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + (abuf ? ACC1_COL : 0u);
#pragma unroll 1
            for (int kb = 0; kb < kblocks; ++kb) {
                // its scales, its codes, and the MMAs that read this slot of
                // tensor memory two items ago: asked for together
                const int s2 = (sslot + SF_STAGES - 2) % SF_STAGES;
                const uint32_t s2_ph = sslot >= 2 ? sph : sph ^ 1u;
                const bool r0 = mbar_try_wait(&sready[sslot], sph), r1 = mbar_try_wait(&full[stage], phase),
                           r2 = item < 2 || mbar_try_wait(&empty[s2], s2_ph);
                if (!__all_sync(0xffffffffu, r0 && r1 && r2) &&
                    !(wait(&sready[sslot], sph) && wait(&full[stage], phase) && (item < 2 || wait(&empty[s2], s2_ph)))) {
                    ok = false;
                    break;
                }
                item = item < 2 ? item + 1 : 2;
                tc_fence_after();
                const uint64_t adesc = smem_desc_k_sw128(smem + OFF_A + stage * A_BYTES);
                const uint64_t bdesc = smem_desc_k_sw128(smem + OFF_B + stage * B_BYTES);
                const uint8_t* sf = smem + OFF_SF + sslot * SF_BYTES;
                const uint32_t slot = tmem_base + SF_COL0 + static_cast<uint32_t>(stage & 1) * SF_STRIDE;
                if (leader) {
#pragma unroll
                    for (int j = 0; j < 6; ++j) tmem_cp_scales(slot + 4 * j, sf + 512 * j);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {          // 4 x 64 elements of K per stage
                        const uint32_t s = slot + 12 * (k >> 1);
                        umma_mxf4_bs(d_tmem, adesc + 2 * k, bdesc + 2 * k, make_idesc_mxf4(BN, 2 * (k & 1)), s, s + 4,
                                     (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    umma_commit(&empty[sslot]);
                }
                __syncwarp();
                if (++sslot == SF_STAGES) { sslot = 0; sph ^= 1u; }
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (leader) umma_commit(&accf[abuf]);
            __syncwarp();
            aph ^= 1u;
            abuf ^= 1;
        }
        if (!ok && leader) {
            umma_commit(drain);
            volatile int no_abort = 0;
            mbar_wait_bounded(drain, 0, &no_abort, nullptr, kDrainTimeoutNs);
        }
        __syncwarp();
    } else if (warp < LOADERS) {
        // ================= epilogue (warps 2..9)
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        auto arrive = [&](uint64_t* bar) {                 // the warp's reads of tensor memory are done
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        int abuf = 0;
        uint32_t fph0 = 0, fph1 = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total_tiles; tile += gridDim.x) {
            const TileInfo ti = decode_tile<BN, 2 * BKB>(tile, p, seg, nseg);
            const GroupDev& g = p.g[0];
            // the tile's biases, an eighth from each warp; the buffer's tile from
            // two tiles back is done with in every warp, which all were here
            // for the tile between
            float* bias_s = reinterpret_cast<float*>(smem + OFF_BIAS) + abuf * BN;
            if (lane < 8) {
                const int i = (warp - 2) * 32 + 4 * lane;
                const float4 v = (g.bias && ti.n0 + i < N)
                    ? __ldg(reinterpret_cast<const float4*>(g.bias + static_cast<size_t>(ti.mat) * N + ti.n0 + i))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(bias_s + i) = v;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            uint32_t& fph = abuf ? fph1 : fph0;
            // (after a wait gave up the warps keep meeting at the barrier above)
            if (ok) ok = warp_wait(&accf[abuf], fph, abort_flag, p.status, p.timeout_ns, lane);
            if (!ok) { abuf ^= 1; continue; }
            fph ^= 1u;
            tc_fence_after();
            const uint32_t acc = lane_base + (abuf ? ACC1_COL : 0u);
            const size_t row0 = static_cast<size_t>(ti.c_row + quad * 32);       // the warp's first row
            const int rows = min(32, ti.rows_left - quad * 32);                  // of them valid (may be negative)
            // 32 bytes (a sector) of the lane's row, at byte `at` of rows of `pitch` bytes
            auto put = [&](size_t pitch, size_t at, const uint32_t* w) {
                if (lane >= rows) return;
                uint8_t* dst = static_cast<uint8_t*>(g.C) + (row0 + lane) * pitch + at;
                if (mp.wide_rows) {
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" :: "l"(dst), "r"(w[0]), "r"(w[1]),
                                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
                } else {
                    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            };
            // Pairs of 32-column chunks; a warp half has two of the four, the
            // first half the overlapping one (the last pair of buffer 0, the
            // first of buffer 1) first.
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int c0 = 2 * ((2 * i + half + (abuf ? 0 : 3)) & 3);
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c0 * 32), r[0]);
                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c0 * 32 + 32), r[1]);
                tmem_ld_wait_regs(r[0]);
                tmem_ld_wait_regs(r[1]);
                arrive(i == 0 ? ovl : &acce[abuf]);
                uint32_t w4[8];                                  // MXFP4: the pair's 64 columns are 32 bytes of a row
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = c0 + u, n = ti.n0 + c * 32;
                    if (rows <= 0 || n >= N) continue;           // (the same for the whole warp)
                    float v[32];
                    const float4* b4 = reinterpret_cast<const float4*>(bias_s + c * 32);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 b = b4[j];
                        v[4 * j + 0] = __uint_as_float(r[u][4 * j + 0]) + b.x;
                        v[4 * j + 1] = __uint_as_float(r[u][4 * j + 1]) + b.y;
                        v[4 * j + 2] = __uint_as_float(r[u][4 * j + 2]) + b.z;
                        v[4 * j + 3] = __uint_as_float(r[u][4 * j + 3]) + b.w;
                    }
                    if (p.silu) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = silu_fast(v[j]);
                    }
                    if constexpr (OUT == MOE_F32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * q + j]);
                            put(4 * static_cast<size_t>(N), 4 * static_cast<size_t>(n + 8 * q), w);
                        }
                    } else if constexpr (OUT == MOE_BF16) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                __nv_bfloat162 t = __floats2bfloat162_rn(v[16 * q + 2 * j], v[16 * q + 2 * j + 1]);
                                w[j] = *reinterpret_cast<uint32_t*>(&t);
                            }
                            put(2 * static_cast<size_t>(N), 2 * static_cast<size_t>(n + 16 * q), w);
                        }
                    } else {
                        uint32_t m = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
                        const uint32_t sb = mxfp4_scale_byte(m);
                        const float inv = mxfp4_inv_scale(sb == 255u ? 127u : sb);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float t[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) t[j] = v[8 * q + j] * inv;
                            w4[4 * u + q] = sb == 255u ? 0u : f32x8_to_e2m1x8(t);
                        }
                        if (lane < rows) mp.y_scales[((row0 + lane) * N + n) / 32] = static_cast<uint8_t>(sb);
                        const size_t pitch = static_cast<size_t>(N) / 2, at = static_cast<size_t>(ti.n0 + c0 * 32) / 2;
                        if (u == 1) put(pitch, at, w4);
                        else if (n + 32 >= N && lane < rows)     // the row's last 32 columns alone
                            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.C) + (row0 + lane) * pitch + at) =
                                make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                }
            }
            abuf ^= 1;
        }
    } else if (warp == RELAY) {
        // ================= scales: every loader's part of a slot is there, made visible to the copies to tensor memory
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
#pragma unroll 1
        for (int tile = blockIdx.x; tile < total_tiles && ok; tile += gridDim.x) {
#pragma unroll 1
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!warp_wait(&sfull[slot], ph, abort_flag, p.status, p.timeout_ns, lane)) { ok = false; break; }
                fence_proxy_async_smem();
                if (lane == 0) mbar_arrive(&sready[slot]);
                if (++slot == SF_STAGES) { slot = 0; ph ^= 1u; }
            }
        }
    } else {
        // ================= scale loaders (warps 10..13): thread i has A row i and weight rows i, 128 + i
        const int i = tid - LOADERS * 32;
        const int kq = K / 32;                           // scale bytes per row, a multiple of 4
        uint32_t* dst0 = reinterpret_cast<uint32_t*>(smem + OFF_SF + 16 * (i & 31) + 4 * (i >> 5));
        auto start = [&](Item& it) {
            it.tile = blockIdx.x;
            it.kb = 0;
            if (it.tile < total_tiles) it.ti = decode_tile<BN, 2 * BKB>(it.tile, p, seg, nseg);
        };
        auto advance = [&](Item& it) {
            if (++it.kb >= kblocks) {
                it.kb = 0;
                it.tile += gridDim.x;
                if (it.tile < total_tiles) it.ti = decode_tile<BN, 2 * BKB>(it.tile, p, seg, nseg);
            }
        };
        // rows and columns past the end read as 2^0 (their codes read as zero)
        auto load = [&](const Item& it, uint32_t (&s)[6]) {
            const int k0 = it.kb * 8;
            const bool two = k0 + 4 < kq;
            auto row = [&](const uint8_t* base, bool ok, uint32_t& lo, uint32_t& hi) {
                if (kq % 8 == 0) {                           // both words of the stage at once
                    const uint2 v = ok ? __ldg(reinterpret_cast<const uint2*>(base + k0)) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    lo = v.x;
                    hi = v.y;
                    return;
                }
                lo = ok ? __ldg(reinterpret_cast<const uint32_t*>(base + k0)) : 0x7F7F7F7Fu;
                hi = ok && two ? __ldg(reinterpret_cast<const uint32_t*>(base + k0 + 4)) : 0x7F7F7F7Fu;
            };
            row(mp.a_scales + static_cast<size_t>(it.ti.a_row + i) * kq, i < it.ti.rows_left, s[0], s[3]);
            const uint8_t* w = mp.w_scales + (static_cast<size_t>(it.ti.mat) * N + it.ti.n0 + i) * kq;
            row(w, it.ti.n0 + i < N, s[1], s[4]);
            row(w + static_cast<size_t>(128) * kq, it.ti.n0 + 128 + i < N, s[2], s[5]);
        };
        Item cur, ahead;
        start(cur);
        start(ahead);
        int slot = 0;
        uint32_t phase = 0;
        bool aborted = false;
        auto store = [&](const uint32_t (&v)[6]) {
            if (!warp_wait(&empty[slot], phase ^ 1u, abort_flag, p.status, p.timeout_ns, lane)) { aborted = true; return; }
            uint32_t* dst = dst0 + slot * (SF_BYTES / 4);
#pragma unroll
            for (int q = 0; q < 6; ++q) dst[q * 128] = v[q];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfull[slot]);
            if (++slot == SF_STAGES) { slot = 0; phase ^= 1u; }
            advance(cur);
        };
        if (kq % 16 == 0) {
            // K a multiple of 512: the words of up to four stages are one
            // 32-byte read, or two 16-byte ones where rows do not start on
            // 32 bytes (the scattered reads are what the loaders spend their
            // time on)
            struct Quad { uint32_t w[3][8]; };
            auto load4 = [&](const Item& it, Quad& v) {
                auto row = [&](const uint8_t* base, bool ok, uint32_t (&w)[8]) {
                    const uint8_t* src = base + it.kb * 8;
                    if (ok && mp.wide_scales) {
                        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                                       "=r"(w[7]) : "l"(src));
                        return;
                    }
                    const uint4 one = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    const uint4 l = ok ? __ldg(reinterpret_cast<const uint4*>(src)) : one;
                    const uint4 h = ok && it.kb + 2 < kblocks ? __ldg(reinterpret_cast<const uint4*>(src) + 1) : one;
                    w[0] = l.x; w[1] = l.y; w[2] = l.z; w[3] = l.w;
                    w[4] = h.x; w[5] = h.y; w[6] = h.z; w[7] = h.w;
                };
                row(mp.a_scales + static_cast<size_t>(it.ti.a_row + i) * kq, i < it.ti.rows_left, v.w[0]);
                const uint8_t* w = mp.w_scales + (static_cast<size_t>(it.ti.mat) * N + it.ti.n0 + i) * kq;
                row(w, it.ti.n0 + i < N, v.w[1]);
                row(w + static_cast<size_t>(128) * kq, it.ti.n0 + 128 + i < N, v.w[2]);
            };
            constexpr int QUADS = LOOKAHEAD / 4;
            Quad ring[QUADS];
            auto fetch = [&](Quad& v) {
                if (ahead.tile >= total_tiles) return;
                load4(ahead, v);
                ahead.kb = min(ahead.kb + 3, kblocks - 1);
                advance(ahead);
            };
#pragma unroll
            for (int j = 0; j < QUADS; ++j) fetch(ring[j]);
#pragma unroll 1
            while (cur.tile < total_tiles && !aborted) {
#pragma unroll
                for (int j = 0; j < QUADS; ++j) {
                    if (cur.tile >= total_tiles || aborted) break;
                    const Quad& v = ring[j];
                    const int n = min(4, kblocks - cur.kb);          // stages of the tile in this read
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < n && !aborted)
                            store({v.w[0][2 * q], v.w[1][2 * q], v.w[2][2 * q], v.w[0][2 * q + 1], v.w[1][2 * q + 1],
                                   v.w[2][2 * q + 1]});
                    if (aborted) break;
                    fetch(ring[j]);
                }
            }
        } else {
            uint32_t ring[LOOKAHEAD][6];
#pragma unroll
            for (int j = 0; j < LOOKAHEAD; ++j)
                if (ahead.tile < total_tiles) { load(ahead, ring[j]); advance(ahead); }
#pragma unroll 1
            while (cur.tile < total_tiles && !aborted) {
#pragma unroll
                for (int j = 0; j < LOOKAHEAD; ++j) {
                    if (cur.tile >= total_tiles || aborted) break;
                    store(ring[j]);
                    if (ahead.tile < total_tiles) { load(ahead, ring[j]); advance(ahead); }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc<TMEM_COLS>(tmem_base);
    }
}

template <int OUT>
cudaError_t launch_out(const Mx4Params& p, cudaStream_t st) {
    auto kernel = mxfp4_matmul_kernel<OUT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ALLOC);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(device_sm_count()), dim3(NUM_THREADS), ALLOC, st, 1, p);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(const moe_mxfp4_shape& s, const uint8_t* a, const uint8_t* a_scales,
                                const int32_t* seg_offsets, const int32_t* seg_mat, const uint8_t* w,
                                const uint8_t* w_scales, const float* bias, void* y, uint8_t* y_scales,
                                int32_t* status, cudaStream_t st) {
    Mx4Params p;
    std::memset(&p, 0, sizeof(p));
    GroupDev& g = p.tc.g[0];
    g.n_mats = s.n_seg;
    g.offsets = seg_offsets;
    g.bias = bias;
    g.C = y;
    g.N = s.n;
    g.K = s.k;
    g.a_rows = s.rows;
    g.seg_mat = seg_mat;
    g.n_weights = s.n_mats;
    p.tc.silu = s.activation == MOE_ACT_SILU;
    p.tc.status = status;
    p.tc.timeout_ns = kWaitTimeoutNs;
    p.a_scales = a_scales;
    p.w_scales = w_scales;
    p.y_scales = y_scales;
    const size_t pitch = static_cast<size_t>(s.n) * (s.out_dtype == MOE_F32 ? 32 : s.out_dtype == MOE_BF16 ? 16 : 4) / 8;
    p.wide_scales = (reinterpret_cast<uintptr_t>(a_scales) | reinterpret_cast<uintptr_t>(w_scales) | (s.k / 32)) % 32 == 0;
    p.wide_rows = (reinterpret_cast<uintptr_t>(y) | pitch) % 32 == 0;
    if (!encode_tma_2d(&p.tc.a_map[0], a, s.rows, s.k / 2, 1, BM) ||
        !encode_tma_2d(&p.tc.a_map[1], a, s.rows, s.k / 2, 1, FEW_ROWS) ||
        !encode_tma_2d(&p.rest_map, a, s.rows, s.k / 2, 1, BM - FEW_ROWS) ||
        !encode_tma_3d(&p.tc.b_map[0], w, s.n_mats, s.n, s.k / 2, 1, BN))
        return cudaErrorInvalidValue;
    if (s.out_dtype == MOE_F32) return launch_out<MOE_F32>(p, st);
    if (s.out_dtype == MOE_BF16) return launch_out<MOE_BF16>(p, st);
    return launch_out<MOE_MXFP4>(p, st);
}

}  // namespace moe
