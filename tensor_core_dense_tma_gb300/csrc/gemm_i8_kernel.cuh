// gemm_i8_kernel.cuh -- the kernels of the 8-bit integer product that read the
// weights as 8-bit codes and widen them on chip: dot products for a few tokens,
// tiles on one CTA, tiles on CTA pairs.  A tile of tokens reads all weights, from
// L2 where another one has just read them.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_kernel.cuh"
#include "ptx_sm103.cuh"

namespace tcdt_i8 {

using tcdt::WaitCtx;

enum WaitSite : int {     // continues tcdt::WaitSite
    kSiteProducer = 21,
    kSiteConvertFull = 22,
    kSiteConvertSlot = 23,
    kSiteMmaSlot = 24,
    kSiteMmaTokens = 25,
    kSiteAccumulator = 26,
};

struct Params {
    int32_t M, N, K;
    int64_t lda, ldb, ldd;
    const int8_t* A;         // dot_kernel only (the other reads through tensor maps)
    const int8_t* B;
    void* D;
    const float* rs;         // [M], [N], [N], or null
    const float* cs;
    const float* bias;
    uint32_t act;
    int32_t splits;          // CTAs (tile_kernel: of a cluster; dot_kernel: warps) that share K
    uint32_t idesc;
    int* status;
    uint64_t timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    int64_t fi_skip_load;    // test builds only: this stage (counted per CTA) gets no tokens
#endif
};

// Programmatic dependent launch: grid_wait returns once the kernel before in
// the stream (which makes the tokens' codes) has finished and its writes are
// visible; grid_release, in that kernel, lets the next one's CTAs start.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// This CTA's tile of tokens: they go over y and z of the grid, as y ends at
// 65535 (8.4 million tokens); the last ones of z may be beyond the last tile.
__device__ __forceinline__ uint32_t token_tile() { return blockIdx.z * gridDim.y + blockIdx.y; }

template <int OUT>
__device__ __forceinline__ void finish_store(const Params& p, float sum, float rs, float cs, float bias, int64_t m,
                                             int64_t n) {
    float v[1] = {sum * (rs * cs) + bias};
    tcdt::ep_act_w<1, tcdt::kEpKeepNan>(p.act, v);
    tcdt::store_elem<OUT>(p.D, m * p.ldd + n, v[0]);
}

// ---------------------------------------------------------------------------
// dot_kernel: at most MT tokens, sums in 32-bit integers
// ---------------------------------------------------------------------------
// A warp computes R channels for all tokens: lane l takes the 16-byte chunks
// l, l + 32, ... of a row of codes, four products an instruction (dp4a), and
// the lanes' sums are added by shuffles; `splits` warps share a row's chunks
// where there are few channels.  The sums are whole numbers: exact and in no
// order.  Bound by the loads under way: 32 warps an SM with up to 4 KB each
// (one token, 8192 x 8192: 12.6 us, 5.3 TB/s; with 16 warps that held the next
// chunks in registers while they computed 14.3 us, with 40 warps 12.9).
constexpr int kDotWarps = 8;

template <int MT, int R, int OUT>
__global__ void __launch_bounds__(kDotWarps * 32, MT <= 2 ? 4 : 2) dot_kernel(const Params p) {
    __shared__ int part[kDotWarps][MT * R];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int split = warp % p.splits, groups = kDotWarps / p.splits;
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * groups + warp / p.splits) * R;
    int acc[MT][R];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[m][r] = 0;
    // rows past the last repeat it: their sums are not stored
    const int8_t* b[R];
    const int8_t* a[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) b[r] = p.B + min(n0 + r, static_cast<int64_t>(p.N - 1)) * p.ldb;
#pragma unroll
    for (int m = 0; m < MT; ++m) a[m] = p.A + min(m, p.M - 1) * p.lda;
    const int chunks = p.K / 16;
    constexpr int kDeep = MT == 1 ? 8 / R : MT == 2 ? 3 : MT == 4 ? 2 : 1;     // chunks of each row in flight
    const int step = p.splits * 32;
    int c = split * 32 + lane;
    int4 w[kDeep][R];
    auto fetch = [&] {
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
            for (int r = 0; r < R; ++r)
                w[d][r] = c + d * step < chunks ? __ldcs(reinterpret_cast<const int4*>(b[r]) + (c + d * step))
                                                : make_int4(0, 0, 0, 0);
    };
    fetch();
    grid_wait();        // the weights do not come from the kernel before, the tokens may
    while (c < chunks) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int at = c + d * step;
            if (at >= chunks) break;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int4 x = *(reinterpret_cast<const int4*>(a[m]) + at);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[m][r] = __dp4a(x.x, w[d][r].x, acc[m][r]);
                    acc[m][r] = __dp4a(x.y, w[d][r].y, acc[m][r]);
                    acc[m][r] = __dp4a(x.z, w[d][r].z, acc[m][r]);
                    acc[m][r] = __dp4a(x.w, w[d][r].w, acc[m][r]);
                }
            }
        }
        c += kDeep * step;
        fetch();
    }
    // the codes after the last whole chunk, a lane each
    const int k = chunks * 16 + lane;
    if (split == 0 && k < p.K) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[m][r] += static_cast<int>(a[m][k]) * static_cast<int>(b[r][k]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int v = acc[m][r];
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
            if (lane == 0) part[warp][m * R + r] = v;
        }
    __syncthreads();
    if (split == 0)
        for (int i = lane; i < MT * R; i += 32) {
            int sum = 0;
            for (int s = 0; s < p.splits; ++s) sum += part[warp + s][i];
            const int m = i / R;
            const int64_t n = n0 + i % R;
            if (m < p.M && n < p.N)
                finish_store<OUT>(p, static_cast<float>(sum), p.rs ? p.rs[m] : 1.f, p.cs ? p.cs[n] : 1.f,
                                  p.bias ? p.bias[n] : tcdt::kNoBias, m, n);
        }
}

// ---------------------------------------------------------------------------
// tile_kernel: tensor cores, the weights' codes widened into tensor memory
// ---------------------------------------------------------------------------
// The transposed product: 128 channels (rows of weights) x BN tokens.  A
// stage is KS codes of each of the 128 rows (8 bits, as they lie in memory)
// and of the BN tokens (fp16).  Four warps read the codes, a thread a row,
// widen them to fp16 pairs and store them into tensor memory as the A operand
// of tcgen05.mma; the tokens are its B operand in shared memory.  Widening
// into tensor memory and not into shared memory keeps the shared-memory
// traffic of a code at two bytes (in by TMA, out to a register); fp16 there
// would add two written and two read by the MMA.
template <int BN_>
struct TileConfig {
    static constexpr int BN = BN_;
    static constexpr int KS = BN <= 64 ? 128 : 64;
    static constexpr int W_BYTES = 128 * KS;
    static constexpr int X_CHUNK = BN * 128;              // 64 fp16 of each token
    static constexpr int STAGE_BYTES = W_BYTES + X_CHUNK * (KS / 64);
    // two CTAs an SM: 113 KB and 256 TMEM columns each
    static constexpr int STAGES = BN == 16 ? 5 : BN == 64 ? 3 : 4;
    static constexpr int SLOT_COLS = KS / 2;              // A operand of a stage: fp16 pairs
    static constexpr int SLOTS = BN <= 64 ? 3 : 4;
    static constexpr int TMEM_COLS = 256;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 256;
    static constexpr int CTAS = 2;
    // groups of four warps widen and finish: two where the epilogue or the MMAs
    // bound (8192 x 1024 weights, 256 tokens: 13.4 us with one, 12.2 with two), one
    // where the weights' stream does (8192 x 8192, 16 tokens: 16.3 us, 16.9 with
    // two); one warp loads, one issues the MMAs
    static constexpr int GROUPS = BN <= 32 ? 1 : 2, WORKERS = 4 * GROUPS;
    static constexpr int THREADS = 32 * (WORKERS + 2);
    static_assert(BN + SLOTS * SLOT_COLS <= TMEM_COLS, "TMEM");
    static_assert(STAGES >= GROUPS && SLOTS >= GROUPS, "a group's step");
    static_assert(BN * 512 <= STAGES * STAGE_BYTES, "partials fit the ring");
};

__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Four codes as two fp16 pairs.  With its sign bit flipped a code c is the
// byte c + 128; below the byte 0x64 it makes the fp16 number 1024 + c + 128,
// and subtracting 1152 leaves c exactly.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));    // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint4 ld_shared_v4u(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_v4f(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at)
                 : "memory");
    return v;
}

// finish_store of four channels of a token, as one store where D's row allows it.
template <int OUT>
__device__ __forceinline__ void finish_store4(const Params& p, const float4& sum, float rs, const float (&cs)[4],
                                              const float (&bias)[4], int64_t m, int64_t n) {
    float v[4] = {sum.x * (rs * cs[0]) + bias[0], sum.y * (rs * cs[1]) + bias[1], sum.z * (rs * cs[2]) + bias[2],
                  sum.w * (rs * cs[3]) + bias[3]};
    tcdt::ep_act_w<4, tcdt::kEpKeepNan>(p.act, v);
    const int64_t at = m * p.ldd + n;
    constexpr int kBytes = OUT == tcdt::kOutF32 ? 16 : 8;
    char* to = static_cast<char*>(p.D) + at * (kBytes / 4);
    if (n + 4 <= p.N && reinterpret_cast<uintptr_t>(to) % kBytes == 0) {
        if constexpr (OUT == tcdt::kOutF32) *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(tcdt::pack2<OUT>(v[0], v[1]), tcdt::pack2<OUT>(v[2], v[3]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < p.N) tcdt::store_elem<OUT>(p.D, at + i, v[i]);
}

// Tokens first, first + step, ... below `cols` of an accumulator, finished and
// stored, a channel a lane: 16 tokens at a time, of which lane i brings token
// i's scale; the activation is chosen once, a warp stores 32 channels of a
// token.  All lanes of the warp take part.
template <int OUT>
__device__ __forceinline__ void store_tokens(const Params& p, uint32_t taddr, int cols, int first, int step, int m0,
                                             int64_t n, float cs, float bias) {
    const int lane = threadIdx.x % 32;
#pragma unroll 1
    for (int c = first; c < cols; c += step) {
        uint32_t acc[16];
        tcdt::tmem_ld_32x32b_x16(taddr + c, acc);
        const int mine = m0 + c + lane % 16;
        const float rs = p.rs && mine < p.M ? p.rs[mine] : 1.f;
        tcdt::tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(acc[i]) * (__shfl_sync(~0u, rs, i) * cs) + bias;
        tcdt::ep_act_w<16, tcdt::kEpKeepNan>(p.act, v);
        const int64_t at = static_cast<int64_t>(m0 + c) * p.ldd + n;
        if (n < p.N) {
            if (c + 16 <= cols) {
#pragma unroll
                for (int i = 0; i < 16; ++i) tcdt::store_elem<OUT>(p.D, at + i * p.ldd, v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols) tcdt::store_elem<OUT>(p.D, at + i * p.ldd, v[i]);
            }
        }
        __syncwarp();      // the next read of tensor memory is the whole warp's
    }
}

// A cluster of p.splits CTAs computes one tile, each a range of the K blocks;
// their partial sums meet in shared memory, and each CTA finishes its share
// of the tokens, adding the partials in the order of their ranges.
template <int BN, int OUT>
__global__ void __launch_bounds__(TileConfig<BN>::THREADS, TileConfig<BN>::CTAS)
tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
    using Cfg = TileConfig<BN>;
    constexpr int KS = Cfg::KS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tcdt::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bar_base = base + Cfg::STAGES * Cfg::STAGE_BYTES;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (Cfg::STAGES + s); };
    auto slot_full = [&](int s) { return bar_base + 8u * (2 * Cfg::STAGES + s); };
    auto slot_empty = [&](int s) { return bar_base + 8u * (2 * Cfg::STAGES + Cfg::SLOTS + s); };
    const uint32_t acc_bar = bar_base + 8u * (2 * Cfg::STAGES + 2 * Cfg::SLOTS);
    const uint32_t drain_bar = acc_bar + 8u;
    static_assert(8 * (2 * Cfg::STAGES + 2 * Cfg::SLOTS + 2) + 8 <= 256, "barriers");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (drain_bar + 8u - raw));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = p.splits > 1 ? static_cast<int>(tcdt::cluster_ctarank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x / p.splits) * 128;
    if (token_tile() * BN >= static_cast<uint32_t>(p.M)) return;     // the whole cluster's
    const int m0 = static_cast<int>(token_tile()) * BN;
    const int blocks = (p.K + KS - 1) / KS;
    const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / p.splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            tcdt::mbar_init(full_bar(s), 1);
            tcdt::mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < Cfg::SLOTS; ++s) {
            tcdt::mbar_init(slot_full(s), 4);
            tcdt::mbar_init(slot_empty(s), 1);
        }
        tcdt::mbar_init(acc_bar, 1);
        tcdt::mbar_init(drain_bar, 1);
        *abort_flag = 0;
        tcdt::fence_mbar_init();
    }
    if (warp == Cfg::WORKERS && lane == 0) {
        tcdt::tma_prefetch_desc(&tmW);
        tcdt::tma_prefetch_desc(&tmX);
    }
    if (warp == Cfg::WORKERS + 1) {
        tcdt::tmem_alloc<1>(tcdt::smem_addr(tmem_slot), Cfg::TMEM_COLS);
        tcdt::tmem_relinquish_alloc_permit<1>();
    }
    tcdt::tc_fence_before_sync();
    __syncthreads();
    tcdt::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{p.status, p.timeout_ns, abort_flag};
    bool ok = true;

    if (warp == Cfg::WORKERS) {
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        // the first weights are on their way before the tokens' codes are there
        const int ahead = min(Cfg::STAGES, kb1 - kb0);
        auto load_tokens = [&](int kb, int to) {
            const uint32_t sx = base + to * Cfg::STAGE_BYTES + Cfg::W_BYTES;
#pragma unroll
            for (int c = 0; c < KS / 64; ++c)
                tcdt::tma_load_2d(sx + c * Cfg::X_CHUNK, &tmX, full_bar(to), kb * KS + 64 * c, m0);
        };
        if (tcdt::elect_one_sync())
            for (int i = 0; i < ahead; ++i) {
                tcdt::mbar_arrive_expect_tx(full_bar(i), Cfg::STAGE_BYTES);
                tcdt::tma_load_2d(base + i * Cfg::STAGE_BYTES, &tmW, full_bar(i), (kb0 + i) * KS, n0);
            }
        __syncwarp();
        grid_wait();
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!tcdt::warp_wait_phase(empty_bar(stage), phase ^ 1u, wctx, kSiteProducer)) {
                ok = false;
                break;
            }
            if (tcdt::elect_one_sync()) {
                if (kb - kb0 >= ahead) {
                    tcdt::mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
                    tcdt::tma_load_2d(base + stage * Cfg::STAGE_BYTES, &tmW, full_bar(stage), kb * KS, n0);
                }
#ifdef TCDT_FAULT_INJECTION
                // the barrier expects bytes that never come: a wait downstream must run out
                if (issued != p.fi_skip_load)
#endif
                    load_tokens(kb, stage);
            }
            __syncwarp();
            ++issued;
            if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
        }
        // The copies started land before this CTA ends, whoever gave up.
        // Stages whose weights alone were asked for get their tokens first,
        // so that their barriers complete.
        for (; issued < ahead; ++issued) {
            if (tcdt::elect_one_sync()) load_tokens(kb0 + issued, stage);
            __syncwarp();
            if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
        }
        for (int i = 0; i < Cfg::STAGES && i < issued; ++i) {
            if (--stage < 0) stage = Cfg::STAGES - 1, phase ^= 1u;
            tcdt::wait_phase_drain(full_bar(stage), phase, 100000000ull);
        }
    } else if (warp == Cfg::WORKERS + 1) {
        int stage = 0, slot = 0;
        uint32_t phase = 0, slot_phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!tcdt::warp_wait_phase(full_bar(stage), phase, wctx, kSiteMmaTokens) ||
                !tcdt::warp_wait_phase(slot_full(slot), slot_phase, wctx, kSiteMmaSlot)) {
                ok = false;
                break;
            }
            tcdt::tc_fence_after_sync();
            const uint32_t sx = base + stage * Cfg::STAGE_BYTES + Cfg::W_BYTES;
            const uint32_t a = tmem + BN + slot * Cfg::SLOT_COLS;
            if (tcdt::elect_one_sync()) {
#pragma unroll
                for (int k = 0; k < KS / 16; ++k)
                    umma_f16_ts(tmem, a + 8 * k,
                                tcdt::smem_desc_sw128(sx + (k / 4) * Cfg::X_CHUNK + (k % 4) * 32, 16u, 1024u), p.idesc,
                                (kb != kb0 || k != 0) ? 1u : 0u);
                tcdt::umma_commit<1>(empty_bar(stage));
                tcdt::umma_commit<1>(slot_empty(slot));
                if (kb + 1 == kb1) tcdt::umma_commit<1>(acc_bar);
            }
            __syncwarp();
            if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
            if (++slot == Cfg::SLOTS) slot = 0, slot_phase ^= 1u;
        }
        if (!ok) {
            if (tcdt::elect_one_sync()) tcdt::umma_commit<1>(drain_bar);
            __syncwarp();
            tcdt::wait_phase_drain(drain_bar, 0, 100000000ull);
        }
    } else {
        const int r = threadIdx.x % 128, group = warp / 4;   // row of weights, lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;    // first lane of the warp's quarter, in bits 16..
        // 16-byte chunk c of row r: 128-byte rows swap chunks by r mod 8, 64-byte rows by r / 2 mod 4
        const uint32_t row = KS == 128 ? r * 128u : r * 64u;
        const uint32_t swap = KS == 128 ? (r & 7) : ((r >> 1) & 3);
        int stage = group, slot = group;
        uint32_t phase = 0, slot_phase = 0;
        for (int kb = kb0 + group; kb < kb1; kb += Cfg::GROUPS) {
            if (!tcdt::warp_wait_phase(full_bar(stage), phase, wctx, kSiteConvertFull)) {
                ok = false;
                break;
            }
            const uint32_t sw = base + stage * Cfg::STAGE_BYTES + row;
            uint4 q[KS / 16];
#pragma unroll
            for (int c = 0; c < KS / 16; ++c) q[c] = ld_shared_v4u(sw + ((c ^ swap) << 4));
            if (!tcdt::warp_wait_phase(slot_empty(slot), slot_phase ^ 1u, wctx, kSiteConvertSlot)) {
                ok = false;
                break;
            }
            tcdt::tc_fence_after_sync();
            const uint32_t a = tmem + lanes + BN + slot * Cfg::SLOT_COLS;
#pragma unroll
            for (int h = 0; h < KS / 64; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    widen4(q[4 * h + c].x, w[8 * c + 0], w[8 * c + 1]);
                    widen4(q[4 * h + c].y, w[8 * c + 2], w[8 * c + 3]);
                    widen4(q[4 * h + c].z, w[8 * c + 4], w[8 * c + 5]);
                    widen4(q[4 * h + c].w, w[8 * c + 6], w[8 * c + 7]);
                }
                tcdt::tmem_st_32x32b_x32(a + 32 * h, w);
            }
            tcdt::tmem_st_wait();
            tcdt::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) tcdt::mbar_arrive(slot_full(slot));
            if ((stage += Cfg::GROUPS) >= Cfg::STAGES) stage -= Cfg::STAGES, phase ^= 1u;
            if ((slot += Cfg::GROUPS) >= Cfg::SLOTS) slot -= Cfg::SLOTS, slot_phase ^= 1u;
        }
        if (ok && kb1 > kb0) {
            ok = tcdt::warp_wait_phase(acc_bar, 0, wctx, kSiteAccumulator);
            tcdt::tc_fence_after_sync();
        }
        grid_wait();     // for the row scales
        const int64_t n = n0 + r;
        const float cs = p.cs && n < p.N ? p.cs[n] : 1.f, bias = p.bias && n < p.N ? p.bias[n] : tcdt::kNoBias;
        if (ok && p.splits == 1) {
            store_tokens<OUT>(p, tmem + lanes, min(BN, p.M - m0), 16 * group, 16 * Cfg::GROUPS, m0, n, cs, bias);
        } else if (p.splits > 1) {
            // partial sums [token][row]; the ring is free, every copy and MMA has finished
            const int cols = min(BN, p.M - m0);
            float* partial = reinterpret_cast<float*>(smem_raw + (base - raw));
#pragma unroll 1
            for (int c = 16 * group; ok && c < cols; c += 16 * Cfg::GROUPS) {
                uint32_t v[16];
                tcdt::tmem_ld_32x32b_x16(tmem + lanes + c, v);
                tcdt::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols) partial[(c + i) * 128 + r] = __uint_as_float(v[i]);
            }
        }
    }
    if (p.splits > 1) {
        __syncwarp();
        tcdt::cluster_sync_all();
        // A warp takes every eighth of this CTA's tokens, a lane four
        // channels of it: 16-byte reads of each partial, two tokens' at once.
        if (warp < Cfg::WORKERS) {
            const int cols = min(BN, p.M - m0);
            const int c0 = cols * rank / p.splits, c1 = cols * (rank + 1) / p.splits;
            const int64_t n = n0 + 4 * lane;
            float cs[4], bias[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[i] = p.cs && n + i < p.N ? p.cs[n + i] : 1.f;
                bias[i] = p.bias && n + i < p.N ? p.bias[n + i] : tcdt::kNoBias;
            }
            for (int c = c0 + warp; c < c1; c += 2 * Cfg::WORKERS) {
                const int d = c + Cfg::WORKERS;
                const bool two = d < c1;
                float4 x = {}, y = {};
                for (int q = 0; q < p.splits; ++q) {
                    const uint32_t at = tcdt::map_to_cta(base + (c * 128 + 4 * lane) * 4, static_cast<uint32_t>(q));
                    const float4 u = ld_cluster_v4f(at), w = two ? ld_cluster_v4f(at + Cfg::WORKERS * 128 * 4) : float4{};
                    x.x += u.x, x.y += u.y, x.z += u.z, x.w += u.w;
                    y.x += w.x, y.y += w.y, y.z += w.z, y.w += w.w;
                }
                finish_store4<OUT>(p, x, p.rs ? p.rs[m0 + c] : 1.f, cs, bias, m0 + c, n);
                if (two) finish_store4<OUT>(p, y, p.rs ? p.rs[m0 + d] : 1.f, cs, bias, m0 + d, n);
            }
        }
        __syncwarp();
        tcdt::cluster_sync_all();       // nobody leaves while its partials may still be read
    }
    tcdt::tc_fence_before_sync();
    __syncthreads();
    if (warp == Cfg::WORKERS + 1) {
        tcdt::tc_fence_after_sync();
        tcdt::tmem_dealloc<1>(tmem, Cfg::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// pair_kernel: 256 channels x 256 tokens on a CTA pair
// ---------------------------------------------------------------------------
// What bounds the tile kernel with many tokens is what an SM can take in from
// L2, about 51 bytes a cycle: 128 channels (8 bits) and 128 tokens (fp16) of 64
// codes are 24 KB for MMAs of 256 cycles.  With cta_group::2 the two CTAs of a
// pair hold half of the tokens each, so that the same 24 KB feed 512 cycles.
// Each CTA widens its own 128 channels into its own tensor memory; the first
// one's MMAs read both.  A stage's shared memory and its columns of tensor
// memory are freed together, by the commit of its MMAs.  8192 x 8192 weights, 512
// tokens: 46 us (640 cycles a stage) to 56 with tiles of 128 x 128 on one CTA.
struct PairConfig {
    static constexpr int BN = 256, KS = 64;
    static constexpr int W_BYTES = 128 * KS, X_BYTES = (BN / 2) * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int STAGES = 8;
    static constexpr int SLOT_COLS = KS / 2;
    static constexpr int TMEM_COLS = 512;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 512;
    static constexpr int GROUPS = 2, WORKERS = 8, THREADS = 32 * (WORKERS + 2);
    static_assert(BN + STAGES * SLOT_COLS <= TMEM_COLS, "TMEM");
};

// Arrival on a barrier of either CTA of the pair.  What it announces is in
// tensor memory, ordered by tcgen05.fence on both sides; no other memory has to
// be released at cluster scope (which takes several hundred cycles a stage).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int OUT>
__global__ void __launch_bounds__(PairConfig::THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
    using Cfg = PairConfig;
    constexpr int KS = Cfg::KS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tcdt::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bar_base = base + Cfg::STAGES * Cfg::STAGE_BYTES;
    auto w_bar = [&](int s) { return bar_base + 8u * s; };                          // weights landed (each CTA's own)
    auto x_bar = [&](int s) { return bar_base + 8u * (Cfg::STAGES + s); };          // both halves of the tokens (first CTA)
    auto slot_bar = [&](int s) { return bar_base + 8u * (2 * Cfg::STAGES + s); };   // both CTAs' channels widened (first CTA)
    auto empty_bar = [&](int s) { return bar_base + 8u * (3 * Cfg::STAGES + s); };  // MMAs done (both)
    const uint32_t acc_bar = bar_base + 8u * 4 * Cfg::STAGES;
    const uint32_t drain_bar = acc_bar + 8u;
    static_assert(8 * (4 * Cfg::STAGES + 2) + 8 <= 512, "barriers");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (drain_bar + 8u - raw));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(tcdt::cluster_ctarank());
    const bool leader = rank == 0;
    const int n0 = static_cast<int>(blockIdx.x) * 128;       // the pair's channels lie side by side
    if (token_tile() * Cfg::BN >= static_cast<uint32_t>(p.M)) return;     // the whole pair's
    const int m0 = static_cast<int>(token_tile()) * Cfg::BN;
    const int blocks = (p.K + KS - 1) / KS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            tcdt::mbar_init(w_bar(s), 1);
            tcdt::mbar_init(x_bar(s), 1);
            tcdt::mbar_init(slot_bar(s), 8);                 // four warps of each CTA
            tcdt::mbar_init(empty_bar(s), 1);
        }
        tcdt::mbar_init(acc_bar, 1);
        tcdt::mbar_init(drain_bar, 1);
        *abort_flag = 0;
        tcdt::fence_mbar_init();
    }
    if (warp == Cfg::WORKERS && lane == 0) {
        tcdt::tma_prefetch_desc(&tmW);
        tcdt::tma_prefetch_desc(&tmX);
    }
    if (warp == Cfg::WORKERS + 1) {
        tcdt::tmem_alloc<2>(tcdt::smem_addr(tmem_slot), Cfg::TMEM_COLS);
        tcdt::tmem_relinquish_alloc_permit<2>();
    }
    tcdt::tc_fence_before_sync();
    tcdt::cluster_sync_all();               // the peer's barriers are there before anything arrives on them
    tcdt::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{p.status, p.timeout_ns, abort_flag};
    bool ok = true;

    if (warp == Cfg::WORKERS) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        const int ahead = min(Cfg::STAGES, blocks);
        auto load_weights = [&](int kb, int to) {
            tcdt::mbar_arrive_expect_tx(w_bar(to), Cfg::W_BYTES);
            tcdt::tma_load_2d(base + to * Cfg::STAGE_BYTES, &tmW, w_bar(to), kb * KS, n0);
        };
        if (tcdt::elect_one_sync())
            for (int i = 0; i < ahead; ++i) load_weights(i, i);
        __syncwarp();
        grid_wait();
        for (int kb = 0; kb < blocks; ++kb) {
            if (!tcdt::warp_wait_phase(empty_bar(stage), phase ^ 1u, wctx, kSiteProducer)) break;
            if (tcdt::elect_one_sync()) {
                if (kb >= ahead) load_weights(kb, stage);
                if (leader) tcdt::mbar_arrive_expect_tx(x_bar(stage), 2 * Cfg::X_BYTES);
#ifdef TCDT_FAULT_INJECTION
                if (issued != p.fi_skip_load)
#endif
                    tcdt::tma_load_2d_pair(base + stage * Cfg::STAGE_BYTES + Cfg::W_BYTES, &tmX,
                                           tcdt::map_to_cta(x_bar(stage), 0), kb * KS, m0 + rank * (Cfg::BN / 2));
            }
            __syncwarp();
            ++issued;
            if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
        }
        // the copies started land before the pair ends, whoever gave up
        int s = stage;
        uint32_t ph = phase;
        for (int i = 0; leader && i < Cfg::STAGES && i < issued; ++i) {
            if (--s < 0) s = Cfg::STAGES - 1, ph ^= 1u;
            tcdt::wait_phase_drain(x_bar(s), ph, 100000000ull);
        }
        for (; issued < ahead; ++issued)
            if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
        for (int i = 0; i < Cfg::STAGES && i < issued; ++i) {
            if (--stage < 0) stage = Cfg::STAGES - 1, phase ^= 1u;
            tcdt::wait_phase_drain(w_bar(stage), phase, 100000000ull);
        }
    } else if (warp == Cfg::WORKERS + 1) {
        if (leader) {
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = 0; kb < blocks; ++kb) {
                if (!tcdt::warp_wait_phase(x_bar(stage), phase, wctx, kSiteMmaTokens) ||
                    !tcdt::warp_wait_phase(slot_bar(stage), phase, wctx, kSiteMmaSlot)) {
                    ok = false;
                    break;
                }
                tcdt::tc_fence_after_sync();
                const uint32_t sx = base + stage * Cfg::STAGE_BYTES + Cfg::W_BYTES;
                const uint32_t a = tmem + Cfg::BN + stage * Cfg::SLOT_COLS;
                if (tcdt::elect_one_sync()) {
#pragma unroll
                    for (int k = 0; k < KS / 16; ++k)
                        umma_f16_ts_pair(tmem, a + 8 * k, tcdt::smem_desc_sw128(sx + k * 32, 16u, 1024u), p.idesc,
                                         (kb != 0 || k != 0) ? 1u : 0u);
                    tcdt::umma_commit<2>(empty_bar(stage), 3);
                    if (kb + 1 == blocks) tcdt::umma_commit<2>(acc_bar, 3);
                }
                __syncwarp();
                if (++stage == Cfg::STAGES) stage = 0, phase ^= 1u;
            }
            if (!ok) {
                if (tcdt::elect_one_sync()) tcdt::umma_commit<2>(drain_bar, 1);
                __syncwarp();
                tcdt::wait_phase_drain(drain_bar, 0, 100000000ull);
            }
        }
    } else {
        const int r = threadIdx.x % 128, group = warp / 4;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;
        int stage = group;
        uint32_t phase = 0;
        for (int kb = group; kb < blocks; kb += Cfg::GROUPS) {
            // (the weights come into a stage whose MMAs are done, so its columns are free too)
            if (!tcdt::warp_wait_phase(w_bar(stage), phase, wctx, kSiteConvertFull)) {
                ok = false;
                break;
            }
            const uint32_t sw = base + stage * Cfg::STAGE_BYTES + r * 64u;
            uint4 q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = ld_shared_v4u(sw + ((c ^ ((r >> 1) & 3)) << 4));
            tcdt::tc_fence_after_sync();
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                widen4(q[c].x, w[8 * c + 0], w[8 * c + 1]);
                widen4(q[c].y, w[8 * c + 2], w[8 * c + 3]);
                widen4(q[c].z, w[8 * c + 4], w[8 * c + 5]);
                widen4(q[c].w, w[8 * c + 6], w[8 * c + 7]);
            }
            tcdt::tmem_st_32x32b_x32(tmem + lanes + Cfg::BN + stage * Cfg::SLOT_COLS, w);
            tcdt::tmem_st_wait();
            tcdt::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(tcdt::map_to_cta(slot_bar(stage), 0));
            if ((stage += Cfg::GROUPS) >= Cfg::STAGES) stage -= Cfg::STAGES, phase ^= 1u;
        }
        if (ok) {
            ok = tcdt::warp_wait_phase(acc_bar, 0, wctx, kSiteAccumulator);
            tcdt::tc_fence_after_sync();
        }
        grid_wait();     // for the row scales
        const int64_t n = n0 + r;
        const float cs = p.cs && n < p.N ? p.cs[n] : 1.f, bias = p.bias && n < p.N ? p.bias[n] : tcdt::kNoBias;
        const int cols = min(Cfg::BN, p.M - m0);
        if (ok) store_tokens<OUT>(p, tmem + lanes, cols, 16 * group, 16 * Cfg::GROUPS, m0, n, cs, bias);
    }
    tcdt::tc_fence_before_sync();
    __syncwarp();
    tcdt::cluster_sync_all();               // the MMAs into the peer's tensor memory are finished
    if (warp == Cfg::WORKERS + 1) {
        tcdt::tc_fence_after_sync();
        tcdt::tmem_dealloc<2>(tmem, Cfg::TMEM_COLS);
    }
}

}  // namespace tcdt_i8
