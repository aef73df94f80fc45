// adapters_kernel.cuh -- the low-rank products of adapters.cu on the tensor cores:
// h = s A X of 128 rows at a time, and the gradients of the factors.
//
// Both read a long operand once (X, or dD) and multiply it by something narrow,
// so both are bound by that operand's stream: tiles are as wide as an MMA is tall
// (128), the narrow side is its N, and the long axis (K, or the rows) is shared by a
// cluster of CTAs whose fp32 sums meet through distributed shared memory, in the
// order of their ranges.  Every wait is bounded as in gemm_kernel.cuh.
#pragma once

#include "gemm_kernel.cuh"

namespace tcdt {

constexpr int kAdapterThreads = 192;                  // producer, MMA and four epilogue warps
// Shared memory of the stages, for two CTAs an SM: with one of twice as much, clusters of
// eight found no eight free SMs together (8192 x 8192, rank 64: 31 us to 66).
constexpr int kAdapterSharedBytes = 96 * 1024;
constexpr int kAdapterMaxStages = 6;
constexpr uint32_t kChunk = 8192;                     // 64 x 64 16-bit elements

// Barriers of the two kernels, in static shared memory.
struct AdapterPipe {
    uint64_t full[kAdapterMaxStages], ready[kAdapterMaxStages], empty[kAdapterMaxStages], acc;
    uint32_t tmem;
    int abort_flag;
};

// empty: arrivals that give a stage back.
__device__ __forceinline__ void adapter_pipe_init(AdapterPipe& q, int stages, uint32_t empty) {
    for (int i = 0; i < stages; ++i) {
        mbar_init(smem_addr(&q.full[i]), 1);
        mbar_init(smem_addr(&q.ready[i]), 4);
        mbar_init(smem_addr(&q.empty[i]), empty);
    }
    mbar_init(smem_addr(&q.acc), 1);
    q.abort_flag = 0;
    fence_mbar_init();
}

// The sum over the CTAs of a cluster, in their order, of what lies at `at` in the
// shared memory of each; the loads of all of them are under way together (one after
// the other they took 0.3 us each).
constexpr int kMaxSplits = 8;

__device__ __forceinline__ float cluster_sum(uint32_t at, int splits) {
    float x[kMaxSplits], v = 0.0f;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits)
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[s]) : "r"(map_to_cta(at, static_cast<uint32_t>(s))));
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits) v += x[s];
    return v;
}

__device__ __forceinline__ float4 cluster_sum4(uint32_t at, int splits) {
    float4 x[kMaxSplits], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[s].x), "=f"(x[s].y), "=f"(x[s].z), "=f"(x[s].w)
                         : "r"(map_to_cta(at, static_cast<uint32_t>(s))));
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits) v.x += x[s].x, v.y += x[s].y, v.z += x[s].z, v.w += x[s].w;
    return v;
}

__device__ __forceinline__ uint16_t adapter_bits(float x, bool bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// h as its two parts; an infinity or a NaN is all in the high one.
__device__ __forceinline__ void adapter_split(float h, bool bf16, uint16_t& high, uint16_t& low) {
    high = adapter_bits(h, bf16);
    const float x = adapter_value(high, bf16);
    low = adapter_bits(isfinite(x) ? h - x : 0.0f, bf16);
}

// What the high part of an fp16 value lost, times 2^11: at most 16 times that, within the type's range.
constexpr float kRestScale = 0x1p-11f;

__device__ __forceinline__ uint16_t adapter_rest(float h, uint16_t high) {
    const float x = adapter_value(high, false);
    return adapter_bits(isfinite(x) ? (h - x) * (1.0f / kRestScale) : 0.0f, false);
}

// Stage and phase of a ring.
struct RingAt {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++stage == stages) stage = 0, phase ^= 1u;
    }
};

// ---------------------------------------------------------------------------
// h = s A X
// ---------------------------------------------------------------------------
struct HiddenArgs {
    CUtensorMap tmX;          // boxes of 64 x 128 rows
    CUtensorMap tmA;          // [adapter][rank][K], boxes of 64 x rr, or [adapter][K][rank], of 64 x 64
    const int32_t* index;
    const float* scale;
    int32_t count, rank, part;
    uint32_t wide;            // 1: hidden is wide (adapters.h)
    int32_t rr;               // the rank in whole 16s
    int32_t per_stage;        // adapters of a stage, whose columns lie side by side:
    int32_t pitch;            // columns from one to the next (rr, or 64 or 128)
    uint32_t a_mn;            // 1: down factors are rank-contiguous
    uint32_t idesc, idesc_one;    // N = per_stage * pitch, and for one adapter rr
    int32_t M, k_steps, splits, stages;
    uint16_t* hidden;
    int64_t ldh;
    uint32_t bf16;
    int* status;
    uint64_t timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    int64_t fi_skip_load;     // test builds only: this step's copies (counted per CTA) do not start
#endif
};

// A stage: two blocks of X and the adapters' of both (8 KB each: 4 of rank 16, 1 of
// rank 64), or, beyond rank 64, one.  (Its two waits and the election cost the
// producer as much as its copies: with one block a stage the loop took 680 cycles a
// block, whatever was in flight.)
__host__ __device__ constexpr int hidden_blocks(int rr) { return rr <= 64 ? 2 : 1; }
constexpr int kHiddenBlock = 128 * 128;      // of X, 64 columns
__host__ __device__ constexpr int hidden_adapter_bytes(int rr) { return rr <= 64 ? 8192 : 16384; }
__host__ __device__ constexpr int hidden_stage_bytes(int rr) {
    return hidden_blocks(rr) * (kHiddenBlock + hidden_adapter_bytes(rr));
}

// A cluster of a.splits CTAs computes 128 rows.  The adapters of a stage have
// columns of their own in tensor memory, up to 128 together, and a row takes those of
// its adapter.  With more adapters than fit a stage, X comes again from L2 with
// the next ones, which use the same columns in their own rows: MMAs that leave the
// other rows as they are.  (An MMA costs some 95 cycles to issue however narrow it is:
// one for all adapters of a stage, not one each.)  8192 x 8192, rank 64, four
// adapters: 30 us (134 MB, 20 at the copy rate); 2048 x 4096, rank 32: 9.5, of which 5
// are start and end; 64 adapters of rank 16 in turn, K = 8192, 145 for 512 to 1024 rows, of rank-contiguous
// factors (one adapter a stage) 311 for 64 to 1024.
__global__ void __launch_bounds__(kAdapterThreads) hidden_tile_kernel(const __grid_constant__ HiddenArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ AdapterPipe q;
    __shared__ int list[128], listed;
    __shared__ uint32_t off[128][4];          // rows that are not of a group's adapters
    __shared__ uint8_t slot[128];             // a row's adapter among those of its group
    __shared__ float factor[128];             // its scale
    __shared__ bool given[128];               // whether it has one
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row0 = static_cast<int>(blockIdx.x / a.splits) * 128;
    constexpr uint32_t kCols = 128;
    const bool bf16 = a.bf16 != 0;

    // (steps of one or two blocks; beyond K both operands read as zeros)
    const int blocks = hidden_blocks(a.rr);
    const int kb0 = a.k_steps * rank / a.splits, kb1 = a.k_steps * (rank + 1) / a.splits;
    auto stage_at = [&](int s) { return base + static_cast<uint32_t>(s * hidden_stage_bytes(a.rr)); };

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&a.tmX);
        tma_prefetch_desc(&a.tmA);
        adapter_pipe_init(q, a.stages, 1);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_addr(&q.tmem), kCols);
        tmem_relinquish_alloc_permit<1>();
    }
    // what is before this kernel in the stream has ended; the product may start
    griddep_wait();
    griddep_launch();
    if (warp == 0) {
        if (lane == 0) {
            // the first blocks of X, before the adapters are known (0.6 us); a tile
            // without adapters waits for them at its end
            for (int i = 0; i < a.stages && i < kb1 - kb0; ++i) {
                mbar_expect_tx(smem_addr(&q.full[i]), blocks * kHiddenBlock);
                for (int b = 0; b < blocks; ++b)
                    tma_load_2d(stage_at(i) + b * kHiddenBlock, &a.tmX, smem_addr(&q.full[i]),
                                64 * ((kb0 + i) * blocks + b), row0);
            }
        }
        __syncwarp();
        AdapterWalk<128> walk;
        walk.load(a.index, a.count, row0, a.M, lane);
        uint32_t m[4];
        int g, n = 0;
        uint32_t rows[4] = {~0u, ~0u, ~0u, ~0u};
        while (walk.next(g, m)) {
            const int at = n % a.per_stage;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                rows[w] = at == 0 ? m[w] : rows[w] & m[w];
                if (!(m[w] >> lane & 1u)) slot[32 * w + lane] = static_cast<uint8_t>(at);
                if (lane == 0) off[n / a.per_stage][w] = rows[w];
            }
            if (lane == 0) list[n] = g;
            ++n;
        }
        if (lane == 0) listed = n;
        __syncwarp();
    }
    if (warp >= 2) {
        // (here, not where they are used: two loads that wait for one another)
        const int row = row0 + static_cast<int>(threadIdx.x) - 64;
        const int g = row < a.M ? __ldg(a.index + row) : -1;
        factor[threadIdx.x - 64] = g < 0 || g >= a.count ? 0.0f : a.scale ? __ldg(a.scale + g) : 1.0f;
        given[threadIdx.x - 64] = g >= 0 && g < a.count;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = q.tmem;
    const int n = warp_uniform<8>(listed);
    const int early = min(a.stages, kb1 - kb0);        // steps whose X is under way
    const int groups = n <= a.per_stage ? (n > 0 ? 1 : 0) : (n + a.per_stage - 1) / a.per_stage;
    const uint32_t a_bytes = a.a_mn ? (a.rr <= 64 ? kChunk : 2 * kChunk) : static_cast<uint32_t>(a.rr) * 128u;
    const WaitCtx wctx{a.status, a.timeout_ns, &q.abort_flag};
    bool ok = true;
    // The order of the steps: the first `early` stages take the first group of
    // adapters of blocks kb0 .., whose X is on its way; then those blocks' other groups,
    // and the other blocks.  (Counted, not divided: two divisions a step were half of the
    // producer's time.)
    const int steps = (kb1 - kb0) * groups;
    struct Step {
        int i = 0, kb, j = 0;
    };
    auto advance = [&](Step& s) {
        if (++s.i < early) {
            ++s.kb;
        } else if (s.i == early && groups > 1) {
            s.kb = kb0, s.j = 1;
        } else if (++s.j >= groups) {
            ++s.kb;
            s.j = groups > 1 && s.kb < kb0 + early ? 1 : 0;
        }
    };

    if (warp == 0) {
        RingAt at;
        int issued = 0;
        if (groups == 0) {
            for (int i = 0; i < early; ++i) {
                if (elect_one_sync()) mbar_arrive(smem_addr(&q.full[i]));
                __syncwarp();
            }
            issued = early;
            for (int i = 0; i < early; ++i) at.next(a.stages);
            ok = false;               // nothing more: wait for them below
        }
        for (Step s{0, kb0, 0}; ok && s.i < steps; advance(s)) {
            if (!warp_wait_phase(smem_addr(&q.empty[at.stage]), at.phase ^ 1u, wctx, kSiteProducerEmpty)) {
                // (the early copies of X land all the same)
                for (int k = s.i; k < early; ++k) {
                    if (elect_one_sync()) mbar_arrive(smem_addr(&q.full[at.stage]));
                    __syncwarp();
                    ++issued;
                    at.next(a.stages);
                }
                ok = false;
                break;
            }
            const uint32_t bar = smem_addr(&q.full[at.stage]), sx = stage_at(at.stage), sa = sx + blocks * kHiddenBlock;
            const int first = s.j * a.per_stage, here = min(a.per_stage, n - first), k0 = 64 * blocks * s.kb;
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(bar, (s.i < early ? 0u : blocks * kHiddenBlock) + blocks * here * a_bytes);
                if (s.i >= early)
                    for (int b = 0; b < blocks; ++b)
                        tma_load_2d(sx + b * kHiddenBlock, &a.tmX, bar, k0 + 64 * b, row0);
#ifdef TCDT_FAULT_INJECTION
                if (issued != a.fi_skip_load)
#endif
                for (int e = 0; e < here; ++e) {
                    const int g = list[first + e];
                    const uint32_t dst = sa + e * a_bytes;
                    for (int b = 0; b < blocks; ++b) {
                        const uint32_t to = dst + b * hidden_adapter_bytes(a.rr);
                        if (a.a_mn) {
                            tma_load_3d(to, &a.tmA, bar, 0, k0 + 64 * b, g);
                            if (a.rr > 64) tma_load_3d(to + kChunk, &a.tmA, bar, 64, k0 + 64 * b, g);
                        } else {
                            tma_load_3d(to, &a.tmA, bar, k0 + 64 * b, 0, g);
                        }
                    }
                }
            }
            __syncwarp();
            ++issued;
            at.next(a.stages);
        }
        if (!ok) {
            // wind down: let the copies already issued land before exiting
            for (int i = 0; i < a.stages && i < issued; ++i) {
                if (--at.stage < 0) at.stage = a.stages - 1, at.phase ^= 1u;
                wait_phase_drain(smem_addr(&q.full[at.stage]), at.phase, 100000000ull);
            }
        }
    } else if (warp == 1) {
        RingAt at;
        const uint32_t lbo = a.a_mn ? kChunk : 16u, kstep = a.a_mn ? 16u * 128u : 32u;
        for (Step s{0, kb0, 0}; s.i < steps; advance(s)) {
            if (!warp_wait_phase(smem_addr(&q.full[at.stage]), at.phase, wctx, kSiteMmaFull)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t sx = stage_at(at.stage), sa = sx + blocks * kHiddenBlock;
            if (elect_one_sync()) {
                const uint32_t m[4] = {off[s.j][0], off[s.j][1], off[s.j][2], off[s.j][3]};
                const uint32_t idesc = n == 1 ? a.idesc_one : a.idesc;
                for (int b = 0; b < blocks; ++b) {
                    const uint32_t xb = sx + b * kHiddenBlock, ab = sa + b * hidden_adapter_bytes(a.rr);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t xdesc = smem_desc_sw128(xb + k * 32u, 16u, 1024u);
                        const uint64_t adesc = smem_desc_sw128(ab + k * kstep, lbo, 1024u);
                        const uint32_t more = s.kb != kb0 || b != 0 || k != 0 ? 1u : 0u;
                        if (groups == 1) umma_f16_ss<1>(tmem, xdesc, adesc, idesc, more);
                        else umma_f16_ss_rows<1>(tmem, xdesc, adesc, idesc, m, more);
                    }
                }
                umma_commit<1>(smem_addr(&q.empty[at.stage]));
            }
            __syncwarp();
            at.next(a.stages);
        }
        if (elect_one_sync()) umma_commit<1>(smem_addr(&q.acc));
        __syncwarp();
        if (!ok) wait_phase_drain(smem_addr(&q.acc), 0, 100000000ull);
    }
    __syncwarp();
    // the four epilogue warps: this CTA's sums of 128 rows, in shared memory, rows 132 numbers apart
    constexpr int kPitch = 128 + 4;
    const int columns = n == 1 ? a.rr : min(n, a.per_stage) * a.pitch;
    float* sums = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)));
    const int t = static_cast<int>(threadIdx.x) - 64;
    if (warp >= 2) {
        ok = warp_wait_phase(smem_addr(&q.acc), 0, wctx, kSiteEpilogueAccFull);
        if (ok && n > 0) {
            tc_fence_after_sync();
            const int quad = warp & 3, row = 32 * quad + lane;
            for (int c = 0; c < columns; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * quad) << 16) + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<uint4*>(sums + row * kPitch + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            }
            tc_fence_before_sync();
        }
        __syncwarp();
    }
    if (a.splits > 1) cluster_sync_all();
    else __syncthreads();
    if (warp >= 2) {
        // this CTA's share of the rows: sums of all ranges in their order, four columns a
        // thread, two times four under way together
        const int rows = 128 / a.splits, quads = a.part / 4, total = rows * quads;
        const int shift = a.part <= 16 ? 2 : a.part <= 32 ? 3 : a.part <= 64 ? 4 : 5;      // of quads
        for (int i0 = t; i0 < total; i0 += 256) {
            float4 sum[2];
            int row[2], c[2];
            bool here[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = i0 + 128 * k;
                here[k] = i < total;
                row[k] = rank * rows + (here[k] ? i >> shift : 0), c[k] = (i & (quads - 1)) * 4;
                sum[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (here[k] && given[row[k]] && c[k] < a.rr) {
                    const uint32_t from = smem_addr(sums + row[k] * kPitch + slot[row[k]] * a.pitch + c[k]);
                    sum[k] = a.splits > 1 ? cluster_sum4(from, a.splits) : ld_shared_v4f(from);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!here[k] || row0 + row[k] >= a.M) continue;
                const float v[4] = {sum[k].x, sum[k].y, sum[k].z, sum[k].w};
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    adapter_split(c[k] + e < a.rank ? v[e] * factor[row[k]] : 0.0f, bf16, hi[e], lo[e]);
                uint16_t* out = a.hidden + (row0 + row[k]) * a.ldh + c[k];
                *reinterpret_cast<uint2*>(out + (a.wide ? a.part : 0)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                *reinterpret_cast<uint2*>(out + (a.wide ? 0 : a.part)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                if (a.wide) {
                    uint32_t rest[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rest[e] = adapter_rest(c[k] + e < a.rank ? v[e] * factor[row[k]] : 0.0f, hi[e]);
                    *reinterpret_cast<uint2*>(out + 2 * a.part) = make_uint2(rest[0] | rest[1] << 16, rest[2] | rest[3] << 16);
                }
            }
        }
    }
    __syncwarp();
    // nobody leaves while its sums may still be read
    if (a.splits > 1) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, kCols);
    }
}

// ---------------------------------------------------------------------------
// gradients of the factors: for an adapter g, sum over its rows of x[i] h[i]^T
// ---------------------------------------------------------------------------
struct FactorArgs {
    CUtensorMap tmX, tmH;     // of each 64 x 64 boxes; tmH's columns are high and low parts
    float low;                // what the low parts count: 1, or 2^-11 of those times 2^11
    void* out;                // element (g, r, c) at out[g * stride + r * sr + c * sc]
    int64_t stride, sr, sc;
    int32_t columns, blocks;  // blocks of 128 columns
};

struct FactorGradArgs {
    FactorArgs f[2];          // down (X and p) and up (dD and h)
    const int32_t* index;
    int32_t rank, part;
    uint32_t idesc;
    int64_t M;
    int32_t splits, stages;
    uint32_t out_kind;        // 0 fp32, 1 fp16, 2 bf16
    int* status;
    uint64_t timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    int64_t fi_skip_load;     // test builds only: as in HiddenArgs
#endif
};

constexpr int kFactorWindow = 1024;       // tiles of 64 rows looked through at once
constexpr int kFactorPitch = 132;         // of the sums in shared memory

__host__ __device__ constexpr int factor_stage_bytes(int part) { return 2 * 8192 + (part <= 32 ? 1 : part / 32) * 8192; }

// A cluster of a.splits CTAs computes the gradient of 128 columns of one factor:
// the 64-row tiles that hold rows of the adapter, in their order, are shared out
// evenly.  Both operands are read as they lie (the sum runs over their rows, so
// both are MN-major).  In a tile that has other rows too, the epilogue warps
// zero those of both operands in shared memory first: zeros in h alone would let an
// infinity in x through.  Both factors of 4096 x 4096 x 4096, rank 16: 16 us (67 MB, 10 at
// the copy rate); 8192 x 4096 x 4096, rank 64, four adapters: 31 (134 MB, 20).
__global__ void __launch_bounds__(kAdapterThreads) factor_grad_kernel(const __grid_constant__ FactorGradArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ AdapterPipe q;
    __shared__ uint8_t holds[kFactorWindow];          // 0: no row of g, 1: some, 2: nothing else
    __shared__ uint16_t list[kFactorWindow];          // tiles with rows of g; bit 15: others too
    __shared__ int listed;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t item = blockIdx.x / a.splits;
    const int blocks = a.f[0].blocks + a.f[1].blocks;
    const int g = static_cast<int>(item / blocks);
    int block = static_cast<int>(item % blocks);
    const int which = block >= a.f[0].blocks ? 1 : 0;
    if (which) block -= a.f[0].blocks;
    const FactorArgs& f = a.f[which];
    const int col0 = 128 * block;
    const int chunks = a.part <= 32 ? 1 : a.part / 32;     // of h
    const uint32_t stage_bytes = static_cast<uint32_t>(factor_stage_bytes(a.part));
    const uint32_t tmem_cols = 2u * static_cast<uint32_t>(a.part);
    if (threadIdx.x == 0) {
        if (a.M > 0) {        // (without rows there are no maps)
            tma_prefetch_desc(&f.tmX);
            tma_prefetch_desc(&f.tmH);
        }
        adapter_pipe_init(q, a.stages, 5);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_addr(&q.tmem), tmem_cols);
        tmem_relinquish_alloc_permit<1>();
    }
    griddep_wait();       // what is before this kernel in the stream has ended
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = q.tmem;
    const WaitCtx wctx{a.status, a.timeout_ns, &q.abort_flag};
    auto stage_at = [&](int s) { return base + static_cast<uint32_t>(s) * stage_bytes; };
    RingAt at;
    bool ok = true;
    int64_t used = 0;                    // stages that this CTA has gone through
    uint32_t mixed = 0;                  // the phases of the `ready` barriers, which tiles with other rows alone use

    for (int64_t w0 = 0; w0 * 64 < a.M; w0 += kFactorWindow) {
        const int tiles = static_cast<int>(min(static_cast<int64_t>(kFactorWindow), (a.M + 63) / 64 - w0));
        // a tile a thread, its 64 entries in loads that are all under way together
        for (int t = threadIdx.x; t < tiles; t += kAdapterThreads) {
            const int64_t row = (w0 + t) * 64;
            const int32_t* from = a.index + row;
            bool any = false, all = true;
            if (row + 64 <= a.M && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
                int4 x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __ldg(reinterpret_cast<const int4*>(from) + i);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    any |= x[i].x == g || x[i].y == g || x[i].z == g || x[i].w == g;
                    all &= x[i].x == g && x[i].y == g && x[i].z == g && x[i].w == g;
                }
            } else {
                const int n = static_cast<int>(min(a.M - row, static_cast<int64_t>(64)));
#pragma unroll 32
                for (int i = 0; i < 64; ++i) {
                    const bool here = i < n && __ldg(from + i) == g;
                    any |= here;
                    all &= here || i >= n;
                }
            }
            holds[t] = any ? all ? 2 : 1 : 0;
        }
        __syncthreads();
        if (warp == 0) {
            int n = 0;
            for (int t0 = 0; t0 < tiles; t0 += 32) {
                const int h = t0 + lane < tiles ? holds[t0 + lane] : 0;
                const uint32_t some = __ballot_sync(0xffffffffu, h != 0);
                if (h) list[n + __popc(some & ((1u << lane) - 1u))] = static_cast<uint16_t>((t0 + lane) | (h == 1 ? 0x8000 : 0));
                n += __popc(some);
            }
            if (lane == 0) listed = n;
        }
        __syncthreads();
        const int found = warp_uniform<11>(listed);
        const int first = found * rank / a.splits, last = found * (rank + 1) / a.splits;
        if (warp == 0) {
            for (int i = first; ok && i < last; ++i) {
                if (!warp_wait_phase(smem_addr(&q.empty[at.stage]), at.phase ^ 1u, wctx, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&q.full[at.stage]), sx = stage_at(at.stage), sh = sx + 2 * kChunk;
                const int row = static_cast<int>((w0 + (list[i] & 0x7FFF)) * 64);
                if (elect_one_sync()) {
                    mbar_arrive_expect_tx(bar, stage_bytes);
#ifdef TCDT_FAULT_INJECTION
                    if (used != a.fi_skip_load)
#endif
                    tma_load_2d(sx, &f.tmX, bar, col0, row);
                    tma_load_2d(sx + kChunk, &f.tmX, bar, col0 + 64, row);
                    for (int c = 0; c < chunks; ++c) tma_load_2d(sh + c * kChunk, &f.tmH, bar, 64 * c, row);
                }
                __syncwarp();
                ++used;
                at.next(a.stages);
            }
        } else if (warp == 1) {
            for (int i = first; ok && i < last; ++i) {
                bool got = warp_wait_phase(smem_addr(&q.full[at.stage]), at.phase, wctx, kSiteMmaFull);
                if (got && list[i] & 0x8000) {
                    got = warp_wait_phase(smem_addr(&q.ready[at.stage]), mixed >> at.stage & 1u, wctx, kSiteMmaFull);
                    mixed ^= 1u << at.stage;
                }
                if (!got) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sx = stage_at(at.stage), sh = sx + 2 * kChunk;
                if (elect_one_sync()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f16_ss<1>(tmem, smem_desc_sw128(sx + k * 2048u, kChunk, 1024u),
                                       smem_desc_sw128(sh + k * 2048u, kChunk, 1024u), a.idesc, used || k ? 1u : 0u);
                    umma_commit<1>(smem_addr(&q.empty[at.stage]));
                }
                __syncwarp();
                ++used;
                at.next(a.stages);
            }
        } else {
            for (int i = first; ok && i < last; ++i) {
                // (every stage is waited for, so that none is mistaken for a later one)
                if (!warp_wait_phase(smem_addr(&q.full[at.stage]), at.phase, wctx, kSiteEpilogueAccFull)) {
                    ok = false;
                    break;
                }
                if (list[i] & 0x8000) {
                    const int row = (static_cast<int>(threadIdx.x) - 64) >> 1;      // two threads a row of 128 bytes a chunk
                    const int64_t at_row = (w0 + (list[i] & 0x7FFF)) * 64 + row;
                    if (at_row < a.M && __ldg(a.index + at_row) != g) {
                        const uint32_t s = stage_at(at.stage) + static_cast<uint32_t>(row) * 128u + (threadIdx.x & 1u) * 64u;
                        for (int c = 0; c < 2 + chunks; ++c)
#pragma unroll
                            for (int b = 0; b < 64; b += 16) st_shared_v4(s + c * kChunk + b, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&q.ready[at.stage]));
                }
                if (lane == 0) mbar_arrive(smem_addr(&q.empty[at.stage]));
                ++used;
                at.next(a.stages);
            }
        }
        __syncwarp();
        __syncthreads();      // the list is done with
    }
    if (warp == 0 && !ok) {
        for (int i = 0; i < a.stages && i < used; ++i) {
            if (--at.stage < 0) at.stage = a.stages - 1, at.phase ^= 1u;
            wait_phase_drain(smem_addr(&q.full[at.stage]), at.phase, 100000000ull);
        }
    }
    if (warp == 1) {
        if (elect_one_sync()) umma_commit<1>(smem_addr(&q.acc));
        __syncwarp();
        if (!ok) wait_phase_drain(smem_addr(&q.acc), 0, 100000000ull);
    }
    __syncwarp();
    // the sums of this CTA's rows, [rank][column], in shared memory
    float* sums = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)));
    if (warp >= 2) {
        ok = ok && warp_wait_phase(smem_addr(&q.acc), 0, wctx, kSiteEpilogueAccFull);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tc_fence_after_sync();
            const int quad = warp & 3;
            float* to = sums + 32 * quad + lane;
            for (int r = 0; r < a.rank; r += 16) {
                uint32_t hi[16], lo[16];
                if (used) {
                    const uint32_t from = tmem + (static_cast<uint32_t>(32 * quad) << 16) + r;
                    tmem_ld_32x32b_x16(from, hi);
                    tmem_ld_32x32b_x16(from + a.part, lo);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (r + i < a.rank)
                        to[(r + i) * kFactorPitch] =
                            used ? fmaf(__uint_as_float(lo[i]), f.low, __uint_as_float(hi[i])) : 0.0f;
            }
            tc_fence_before_sync();
        }
        __syncwarp();
    }
    if (a.splits > 1) cluster_sync_all();
    else __syncthreads();
    // joined and stored, an equal share by each CTA: eight elements that are neighbours in
    // memory a thread (of a row of d_down, of a column's values in d_up), in 16-byte stores
    // where they can be
    const bool by_rank = f.sr == 1 && f.sc != 1;
    const int total = by_rank ? (a.rank + 7) / 8 * 128 : a.rank * 16, share = (total + a.splits - 1) / a.splits;
    const int esz = a.out_kind == 0 ? 4 : 2;
    const bool units = ((reinterpret_cast<uintptr_t>(f.out) | static_cast<uintptr_t>(f.stride * esz) |
                         static_cast<uintptr_t>((by_rank ? f.sc : f.sr) * esz)) & 15) == 0;
    for (int i = rank * share + threadIdx.x; i < min(total, (rank + 1) * share); i += kAdapterThreads) {
        const int r = by_rank ? i / 128 * 8 : i / 16, c = by_rank ? i % 128 : i % 16 * 8;
        const int n = by_rank ? min(8, a.rank - r) : min(8, f.columns - col0 - c);
        if (col0 + c >= f.columns) continue;
        const uint32_t from = smem_addr(sums + r * kFactorPitch + c);
        float v[8];
        if (by_rank) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t at_e = from + (e < n ? e : 0) * (kFactorPitch * 4u);
                v[e] = a.splits > 1 ? cluster_sum(at_e, a.splits) : ld_shared_f32(at_e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 x = a.splits > 1 ? cluster_sum4(from + 4u * e, a.splits) : ld_shared_v4f(from + 4u * e);
                v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
            }
        }
        const int64_t o = g * f.stride + r * f.sr + (col0 + c) * f.sc, step = by_rank ? f.sr : f.sc;
        if (a.out_kind == 0) {
            float* out = static_cast<float*>(f.out) + o;
            if (units && n == 8) {
                reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) out[e * step] = v[e];
            }
        } else {
            uint16_t* out = static_cast<uint16_t*>(f.out) + o;
            uint16_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = adapter_bits(v[e], a.out_kind == 2);
            if (units && n == 8) {
                *reinterpret_cast<uint4*>(out) = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16,
                                                            x[6] | x[7] << 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) out[e * step] = x[e];
            }
        }
    }
    __syncwarp();
    if (a.splits > 1) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, tmem_cols);
    }
}

}  // namespace tcdt
