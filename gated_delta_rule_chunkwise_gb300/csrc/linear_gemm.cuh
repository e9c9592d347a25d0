// The matrix product behind ldn_linear, ldn_linear_e4m3 and ldn_linear_backward on the 5th-generation
// tensor cores, with its epilogue.
//
//   out[j][i] = epilogue(sum_k A[i][k] B[j][k])
//
// i, the contiguous index of the output, is the lane of tensor memory and j its column, so that a warp
// of the epilogue reads and writes 32 neighbours of a row and a feature's bias is its lane's.  For the
// forward A is the weight and B the tokens; few tokens are then a narrow tile (16 columns and more) of
// full lanes, and the weight streams through once.  For the gradients A is the weight or x transposed
// and B dz: "MN-major" operands, whose contiguous index is i or j, are taken as they lie in memory.
//
// A block takes 128 x BN of the output: one warp issues the TMA loads of 128-byte wide k blocks, one
// thread the products, eight warps the epilogue of the tile before, out of the other half of tensor
// memory.  Few tiles: `split` blocks of a cluster share a tile's k blocks, add their parts through
// distributed shared memory in a fixed order and take a share of the columns each.
//
// The tensor cores cut off what an addition to their accumulators rounds away (an fp32 sum over 4096
// was 4.5e-6 of its norm off, twice that over 8192).  Where the output keeps such digits (PROMOTE: fp32
// outputs) the sum is taken over chunks of k, whose results are added in registers, rounded to nearest.
//
// fp32 inputs come as planes of bf16 (linear_prep.cu): a chunk then runs over pairs of planes, the
// smallest products first.
#pragma once
#include "linear_common.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace ldn {
namespace linear {

using namespace sm100;

constexpr int kLanes = 128, kEpilogue = 256, kThreads = 64 + kEpilogue;
constexpr long long kWaitCycles = 4000000000ll;   // 2 s

// A tile's place in shared memory: 128-byte wide blocks of A, then of B.
template <int BN> struct Tile {
    static constexpr int kABytes = kLanes * 128, kBBytes = BN * 128, kStage = kABytes + kBBytes;
    static constexpr int kStages = 204800 / kStage < 10 ? 204800 / kStage : 10;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr int kTmemCols = 2 * BN;   // two accumulators, a power of two of at least 32
};

__device__ __forceinline__ float gelu(float z)
{
    float bell;
    return z * normal_integral(z, bell);
}

__device__ __forceinline__ float widened(float x) { return x; }
__device__ __forceinline__ float widened(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// f(type) with the element type of `f32`: a branch for the whole warp around N accesses.
template <typename F> __device__ __forceinline__ void with_type(int f32, F f)
{
    if (f32) f(float());
    else f(__nv_bfloat16());
}

// N columns of lane i, from column j on, of which `valid` are there (WHOLE: all, and no access waits
// for a comparison).
template <bool EPI, bool F8, int N, bool WHOLE>
__device__ __forceinline__ void finish_as(const Args &a, float *v, long long i, long long j, int valid)
{
    const long long at = j * a.ni + i;
    if constexpr (EPI) {
        float r[N];
        if (a.residual)   // on its way while the rest is formed
            with_type(a.out_f32, [&](auto e) {
                const decltype(e) *p = (const decltype(e) *)a.residual + at;
#pragma unroll
                for (int c = 0; c < N; ++c, p += a.ni) r[c] = WHOLE || c < valid ? widened(*p) : 0.f;
            });
        if constexpr (F8) {
            const float si = a.scale_i[i];
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] *= si * a.scale_j[j + (WHOLE ? c : min(c, valid - 1))];
        }
        if (a.bias) {
            float b;
            with_type(a.bias_f32, [&](auto e) { b = widened(((const decltype(e) *)a.bias)[i]); });
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] += b;
        }
        if (a.z)
            with_type(a.z_f32, [&](auto e) {
                decltype(e) *p = (decltype(e) *)a.z + at;
#pragma unroll
                for (int c = 0; c < N; ++c, p += a.ni)
                    if (WHOLE || c < valid) put(p, v[c]);
            });
        if (a.activation == LDN_ACT_SILU) {
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] *= sigmoid_fast(v[c]);
        } else if (a.activation == LDN_ACT_GELU) {
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] = gelu(v[c]);
        }
        if (a.residual)
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] += r[c];
    }
    with_type(a.out_f32, [&](auto e) {
        decltype(e) *p = (decltype(e) *)a.out + at;
#pragma unroll
        for (int c = 0; c < N; ++c, p += a.ni)
            if (WHOLE || c < valid) put(p, v[c]);
    });
}

template <bool EPI, bool F8, int N>
__device__ __forceinline__ void finish(const Args &a, float *v, long long i, long long j, int most = N)
{
    if (i >= a.ni || j >= a.nj || most <= 0) return;
    if (most >= N && a.nj - j >= N) finish_as<EPI, F8, N, true>(a, v, i, j, N);
    else finish_as<EPI, F8, N, false>(a, v, i, j, (int)min(a.nj - j, (long long)most));
}

// Tiles in the order that blocks take them: groups of 16 tiles of lanes, through all columns, so that
// the tiles in flight share operands in L2.
struct Place { int mi, nj; };
__device__ __forceinline__ Place place_of(long long t, int mt, int nt)
{
    constexpr int G = 16;
    const long long per = (long long)G * nt;
    const int g = (int)(t / per), rest = (int)(t - g * per), width = min(G, mt - g * G);
    return {g * G + rest % width, rest / width};
}

// A place in the ring of stages, and how often it went round.
template <int STAGES> struct Ring {
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step()
    {
        if (++s == STAGES) {
            s = 0;
            ++round;
        }
    }
};

// mbar_wait without the hint that lets a waiting thread sleep: waking it cost a block of 64 k blocks
// 1 us of 11.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity)
{
    auto passed = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (passed()) return true;
    const long long t0 = clock64();
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (passed()) return true;
    } while (clock64() - t0 < kWaitCycles);
    return false;
}

// Columns c, c + 1, ... of this warp's lanes of tensor memory.
template <int C> __device__ __forceinline__ void load_columns(uint32_t at, float *v)
{
    if constexpr (C == 8) tmem_ld8(at, v);
    else
#pragma unroll
        for (int q = 0; q < C; q += 16) tmem_ld16(at + q, v + q);
    tmem_ld_wait();
}

template <int BN, bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Args a)
{
    using S = Tile<BN>;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[S::kStages], empty[S::kStages], done[2], drained[2], drain;
    __shared__ uint32_t tmem;
    __shared__ int fail;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int split = a.split;
    const uint32_t rank = split > 1 ? cluster_ctarank() : 0;
    constexpr int kElems = F8 ? 128 : 64;   // elements of a k block
    const int mt = (int)((a.ni + kLanes - 1) / kLanes), nt = (int)((a.nj + BN - 1) / BN);
    const long long tiles = (long long)mt * nt, first = blockIdx.x / split, step = gridDim.x / split;
    // this block's k blocks: all, or its share
    const int b0 = (int)((long long)a.kblocks * rank / split), b1 = (int)((long long)a.kblocks * (rank + 1) / split);

    const bool one = elect_one();   // one thread of a warp, the same throughout
    if (warp == 0 && one) {
        fail = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&drained[i], kEpilogue);
        }
        mbar_init(&drain, 1);
        fence_mbar_init();
    }
    if (warp == 2 && one) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 1) {
        tmem_alloc(&tmem, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem;
    Ring<S::kStages> ring;   // of this thread's loads or products

    if (warp == 0 && one) {
        // ---- loads
        bool go = true;
        for (long long t = first; go && t < tiles; t += step) {
            const Place p = place_of(t, mt, nt);
            for (int c0 = b0; go && c0 < b1; c0 += a.chunk) {
                const int c1 = min(b1, c0 + a.chunk);
                for (int pair = 0; go && pair < a.npairs; ++pair) {
                    const int pa = (int)(a.pairs_a >> (4 * pair)) & 15, pb = (int)(a.pairs_b >> (4 * pair)) & 15;
                    for (int k = c0; k < c1; ++k, ring.step()) {
                        const int s = ring.s, at = k * kElems;
                        if (!wait(&empty[s], (ring.round & 1u) ^ 1u)) {
                            fail = 1;
                            go = false;
                            break;
                        }
                        uint8_t *da = sm + s * S::kStage, *db = da + S::kABytes;
                        mbar_arrive_expect_tx(&full[s], S::kStage);
                        if constexpr (AMN) {
#pragma unroll
                            for (int b = 0; b < kLanes / 64; ++b)
                                tma_load_3d(da + b * 8192, &map_a, &full[s], p.mi * kLanes + 64 * b, at, pa);
                        } else {
                            tma_load_3d(da, &map_a, &full[s], at, p.mi * kLanes, pa);
                        }
                        if constexpr (BMN) {
#pragma unroll
                            for (int b = 0; b < BN / 64; ++b)
                                tma_load_3d(db + b * 8192, &map_b, &full[s], p.nj * BN + 64 * b, at, pb);
                        } else {
                            tma_load_3d(db, &map_b, &full[s], at, p.nj * BN, pb);
                        }
                    }
                }
            }
        }
    } else if (warp == 1 && one) {
        // ---- products
        constexpr uint32_t idesc = idesc_f16kind_f32(kLanes, BN, AMN, BMN, F8 ? kMmaE4M3 : kMmaBF16);
        const uint32_t at = smem_u32(sm);
        const uint64_t desc_a = AMN ? mnmajor_desc(at, 64, 0) : kmajor_desc(at, kLanes, 0),
                       desc_b = BMN ? mnmajor_desc(at + S::kABytes, 64, 0) : kmajor_desc(at + S::kABytes, BN, 0);
        int turn = 0;
        bool go = true;
        for (long long t = first; go && t < tiles; t += step)
            for (int c0 = b0; go && c0 < b1; c0 += a.chunk, ++turn) {
                const int acc = turn & 1, n = (min(b1, c0 + a.chunk) - c0) * a.npairs;
                if (!wait(&drained[acc], ((uint32_t)(turn >> 1) & 1u) ^ 1u)) {
                    fail = 1;
                    go = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tbase + acc * BN;
                for (int k = 0; k < n; ++k, ring.step()) {
                    const int s = ring.s;
                    if (!wait(&full[s], ring.round & 1u)) {
                        fail = 1;
                        go = false;
                        break;
                    }
                    tc_fence_after();
                    // a stage and a step of 32 bytes of k further: 16-byte units in the low bits
                    const uint64_t sa = desc_a + s * (S::kStage / 16), sb = desc_b + s * (S::kStage / 16);
#pragma unroll
                    for (uint32_t q = 0; q < 4; ++q) {
                        const uint64_t da = sa + q * (AMN ? 128 : 2), db = sb + q * (BMN ? 128 : 2);
                        if constexpr (F8) umma_f8(d, da, db, idesc, k > 0 || q > 0);
                        else umma_bf16(d, da, db, idesc, k > 0 || q > 0);
                    }
                    umma_commit(&empty[s]);
                }
                if (go) umma_commit(&done[acc]);
            }
    } else if (warp >= 2) {
        // ---- epilogue: this warp's 32 lanes and half of the columns
        constexpr int H = BN / 2, C = H < 32 ? H : 32;
        const uint32_t quad = warp & 3, half = (uint32_t)(warp - 2) >> 2;
        float *part = (float *)sm;   // a split tile's parts, once every stage is free
        int turn = 0;
        bool go = true;
        for (long long t = first; go && t < tiles; t += step) {
            const Place p = place_of(t, mt, nt);
            const long long i = (long long)p.mi * kLanes + quad * 32 + lane, j = (long long)p.nj * BN + half * H;
            // columns [c, c + C) of this half, done
            auto leave = [&](float *v, int c) {
                if (split == 1) {
                    finish<EPI, F8, C>(a, v, i, j + c);
                } else {
#pragma unroll
                    for (int q = 0; q < C; ++q) part[(half * H + c + q) * kLanes + quad * 32 + lane] = v[q];
                }
            };
            float sum[PROMOTE ? H : 1];
            if constexpr (PROMOTE)
#pragma unroll
                for (int c = 0; c < H; ++c) sum[c] = 0.f;
            for (int c0 = b0; c0 < b1; c0 += a.chunk, ++turn) {
                const int acc = turn & 1;
                if (!wait(&done[acc], (uint32_t)(turn >> 1) & 1u)) {
                    fail = 1;
                    go = false;
                    break;
                }
                tc_fence_after();
                const uint32_t row = tbase + (quad << 21) + acc * BN + half * H;
                if constexpr (PROMOTE) {
#pragma unroll
                    for (int c = 0; c < H; c += C) {
                        float v[C];
                        load_columns<C>(row + c, v);
#pragma unroll
                        for (int q = 0; q < C; ++q) sum[c + q] += v[q];
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < H; c += C) {
                        float v[C];
                        load_columns<C>(row + c, v);
                        leave(v, c);
                    }
                }
                tc_fence_before();
                mbar_arrive(&drained[acc]);
            }
            if constexpr (PROMOTE)
                if (go)
#pragma unroll
                    for (int c = 0; c < H; c += C) leave(sum + c, c);
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        constexpr int U = 8;   // columns at a time: as many reads of each block are on their way together
        const uint32_t quad = warp & 3, half = (uint32_t)(warp - 2) >> 2;
        const int mine = BN / 2 / split;   // columns of a half of this block's share
        const Place p = place_of(first, mt, nt);
        const long long i = (long long)p.mi * kLanes + quad * 32 + lane, j = (long long)p.nj * BN;
        const uint32_t at = smem_u32(sm) + (quad * 32 + lane) * 4;
        const int c0 = (rank * 2 + half) * mine, c1 = warp >= 2 ? (int)min((long long)c0 + mine, a.nj - j) : c0;
        // Only what is stored is read: a store waits for its value, so no read is under way when this
        // block says that the others may leave.
        if (i < a.ni)
#pragma unroll 1
            for (int c = c0; c < c1; c += U) {
                float v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = 0.f;
#pragma unroll 2
                for (int q = 0; q < split; ++q) {
                    const uint32_t from = mapa_shared(at, q);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c + u < c1) v[u] += __uint_as_float(ld_shared_cluster_u32(from + (c + u) * kLanes * 4));
                }
                finish<EPI, F8, U>(a, v, i, j + c, c1 - c);
            }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (fail) {
        // what is under way ends before the memory it uses is given back (bounded)
        if (warp == 1 && one) {
            umma_commit(&drain);
            wait(&drain, 0);
        }
        if (warp == 0 && one) {
            atomicOr(a.status, 1 << LDN_ERR_TIMEOUT);
            for (int s = 0; s < S::kStages; ++s)
            {
                const uint32_t loads = ring.round + (s < ring.s);   // that went into stage s
                if (loads) wait(&full[s], (loads - 1) & 1u);
            }
        }
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tbase, S::kTmemCols);
}

}  // namespace linear
}  // namespace ldn
