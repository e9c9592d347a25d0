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
// A block takes 128 x bn of the output: one warp issues the TMA loads of 128-byte wide k blocks, one
// thread the products, eight warps the epilogue of the tile before, out of the other half of tensor
// memory.  Many tiles (PAIR): two blocks of a cluster take 256 x bn together, each loading its half of
// either operand, so that a product's operands cross into an SM once for twice the output.  Few tiles:
// `split` blocks of a cluster share a tile's k blocks; each sends its part of every column to the block
// whose share the column is, by bulk copies between their shared memories, and that one adds the parts in a
// fixed order (128 columns among 4 blocks: 5 us by single stores there, 3 by single reads).
//
// The tensor cores cut off what an addition to their accumulators rounds away (an fp32 sum over 4096
// was 4.5e-6 of its norm off, twice that over 8192).  Where the output would show it (PROMOTE: fp32 outputs,
// and bf16 ones of more than 65536 products) the sum is taken over chunks of k, whose results are added in
// registers, rounded to nearest.
//
// Results leave through shared memory (`staged`), 128 lanes x 32 columns at a time, by TMA stores; bf16
// ones are written there transposed, as fragments of 8 x 8.  Written by the lanes, 2 bytes each, they hold
// the products up (8192 x 512 to 4096: 44 us for 31).  A residual comes in the same way, into the place of
// the results, while the products run (as loads of the lanes: 8192 x 4096 to 4096 with fp32, 220 us).
//
// fp32 inputs come as planes of bf16 (linear_prep.cu): a chunk then runs over pairs of planes, the
// smallest products first.
#pragma once
#include "linear_common.cuh"
#include "linear_plan.h"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace ldn {
namespace linear {

using namespace sm100;

constexpr int kLanes = 128, kEpilogue = 256, kThreads = 64 + kEpilogue;
constexpr long long kWaitCycles = 4000000000ll;   // 2 s

// A block's stages in shared memory: 128-byte wide blocks of A, then of B, at multiples of 1024 bytes.
constexpr int kABytes = kLanes * 128, kMostStages = 10, kStageBytes = 224 * 1024;   // with what follows them
__host__ __device__ inline int stage_bytes(int columns) { return kABytes + columns * 128; }   // of B in this block
// Two pairs of buffers for each half of the epilogue's warps, one filled while the other is read.  A buffer
// is 32 columns of 128 lanes in bf16, as two boxes of 64, or half of 32 columns in fp32.
constexpr int kBuffer = 32 * kLanes * 2, kStaging = 8 * kBuffer;
// Room for the parts of a split tile: bn columns of 128 lanes.
__host__ __device__ inline int part_bytes(int bn, int split) { return split > 1 ? bn * kLanes * 4 : 0; }

// N values through an activation.
template <int N> __device__ __forceinline__ void activate(float *v, int activation)
{
    if (__builtin_expect(activation == LDN_ACT_SILU, 0)) {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 y = silu_fast(make_float2(v[c], v[c + 1]));
            v[c] = y.x;
            v[c + 1] = y.y;
        }
    } else if (__builtin_expect(activation == LDN_ACT_GELU, 0)) {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 y = gelu(make_float2(v[c], v[c + 1]));
            v[c] = y.x;
            v[c + 1] = y.y;
        }
    }
}

// 16 columns of lane i, from column j on, of which `valid` are there.  There is one copy of this code in a
// kernel and no other for whole chunks: what a small product executes once comes from a cold instruction
// cache.
// z, stored where it is wanted, and the activation.
template <bool EPI, bool F8>
__device__ __forceinline__ void apply16(const Args &a, float *v, long long i, long long j, int valid)
{
    if constexpr (EPI) {
        if (valid <= 0 || i >= a.ni) return;
        if constexpr (F8) {
            const float si = a.scale_i[i];
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] *= si * a.scale_j[j + min(c, valid - 1)];
        }
        if (a.bias) {
            const float b = a.bias_f32 ? ((const float *)a.bias)[i] : __bfloat162float(((const __nv_bfloat16 *)a.bias)[i]);
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] += b;
        }
        if (a.z) {
            const long long at = j * a.ni + i;
            if (a.z_f32)
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    if (c < valid) ((float *)a.z)[at + c * a.ni] = v[c];
                }
            else
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (c < valid) ((__nv_bfloat16 *)a.z)[at + c * a.ni] = __float2bfloat16_rn(v[c]);
        }
        activate<16>(v, a.activation);
    }
}
// The residual, and the result.
template <bool EPI>
__device__ __forceinline__ void store16(const Args &a, float *v, long long i, long long j, int valid)
{
    if (valid <= 0 || i >= a.ni) return;
    const long long at = j * a.ni + i;
    if (EPI && a.residual) {
        float r[16];
        if (a.out_f32)
#pragma unroll
            for (int c = 0; c < 16; ++c) r[c] = ((const float *)a.residual)[at + min(c, valid - 1) * a.ni];
        else
#pragma unroll
            for (int c = 0; c < 16; ++c)
                r[c] = __bfloat162float(((const __nv_bfloat16 *)a.residual)[at + min(c, valid - 1) * a.ni]);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] += r[c];
    }
    if (a.out_f32) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < valid) ((float *)a.out)[at + c * a.ni] = v[c];
    } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < valid) ((__nv_bfloat16 *)a.out)[at + c * a.ni] = __float2bfloat16_rn(v[c]);
    }
}

// Tiles in the order that blocks take them: groups of about 2048 lanes, through all columns, so that
// the tiles in flight share operands in L2.
// (A product of at most 2^40 elements has fewer than 2^30 tiles: 32-bit divisions, 64-bit ones of three
// roles took a call 1 us.)
struct Place { int mi, nj; };
__device__ __forceinline__ Place place_of(unsigned t, unsigned mt, unsigned nt, unsigned group)
{
    const unsigned per = group * nt, g = t / per, width = min(group, mt - g * group), rest = t - g * per;
    return {(int)(g * group + rest % width), (int)(rest / width)};
}

// A place in the ring of stages, and how often it went round.
struct Ring {
    int stages, s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step()
    {
        if (++s == stages) {
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
#pragma unroll
    for (int q = 0; q < C; q += 16) tmem_ld16(at + q, v + q);
    tmem_ld_wait();
}

template <bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
            const __grid_constant__ CUtensorMap map_residual, const Args a)
{
    extern __shared__ uint8_t raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kMostStages], empty[kMostStages], done[2], drained[2], loaded[4], met, drain;
    __shared__ uint32_t tmem;
    __shared__ int fail;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const bool one = elect_one();   // one thread of a warp, the same throughout
    const int split = PAIR ? 1 : a.split, bn = a.bn, stages = a.stages, cols = PAIR ? bn / 2 : bn,
              stage = stage_bytes(cols);
    const uint32_t rank = PAIR || split > 1 ? cluster_ctarank() : 0;
    constexpr int kElems = F8 ? 128 : 64;                  // elements of a k block
    constexpr int kTileLanes = PAIR ? 2 * kLanes : kLanes;
    const int mt = (int)((a.ni + kTileLanes - 1) / kTileLanes), nt = (int)((a.nj + bn - 1) / bn);
    constexpr int kGroup = 2048 / kTileLanes;
    const int blocks = PAIR ? 2 : split;                   // that share a tile
    const unsigned tiles = (unsigned)mt * nt, first = blockIdx.x / (unsigned)blocks, step = gridDim.x / (unsigned)blocks;
    // this block's k blocks: all, or its share
    const int b0 = PAIR ? 0 : (int)((unsigned)a.kblocks * rank / split),
              b1 = PAIR ? a.kblocks : (int)((unsigned)a.kblocks * (rank + 1) / split);
    const uint32_t tcols = tensor_columns(bn, PROMOTE);    // two accumulators

    if (warp == 0 && one) {
        fail = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&drained[i], (PAIR ? 2 : 1) * (kEpilogue / 32));
            mbar_init(&loaded[i], 1);
            mbar_init(&loaded[2 + i], 1);
        }
        mbar_init(&drain, 1);
        mbar_init(&met, 1);
        fence_mbar_init();
        if (!PAIR && split > 1) mbar_arrive_expect_tx(&met, part_bytes(bn, split));
    }
    if (warp == 2 && one) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(&tmem, tcols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem, tcols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (PAIR) {
        cluster_sync();   // the other block's barriers are there
    } else {
        // the loads need nothing but the barriers, which their own thread made
        __syncwarp();
        if (warp == 0) named_arrive(1, kThreads);
        else named_sync(1, kThreads);
        if (split > 1) cluster_arrive_relaxed();
    }
    tc_fence_after();
    const uint32_t tbase = warp == 0 ? 0 : tmem;
    griddep_wait();   // what was set up so far touches no memory of another kernel
    griddep_launch_dependents();
    Ring ring{stages};   // of this thread's loads or products
    // this warp has read accumulator acc
    auto drained_by = [&](int acc) {
        tc_fence_before();
        __syncwarp();
        if (one) {
            if constexpr (PAIR) mbar_remote_arrive(mapa_shared(smem_u32(&drained[acc]), 0));
            else mbar_arrive(&drained[acc]);
        }
    };
    // a half's columns of a split tile's share: multiples of 16, or all for the first
    auto per_half = [](int share, uint32_t half, int &h0, int &h) {
        const int per = (share / 2 + 15) & ~15;
        h0 = half * per;
        h = max(0, min(per, share - h0));
    };

    if (warp == 0 && one) {
        // ---- loads
        bool go = true;
        for (unsigned t = first; go && t < tiles; t += step) {
            const Place p = place_of(t, mt, nt, kGroup);
            const int ia = p.mi * kTileLanes + (PAIR ? rank * kLanes : 0), jb = p.nj * bn + (PAIR ? rank * cols : 0);
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
                        uint8_t *da = sm + s * stage, *db = da + kABytes;
                        // a pair's bytes are all counted on the first block's barrier
                        if (!PAIR || rank == 0) mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * stage);
                        const uint32_t bar = PAIR ? mapa_shared(smem_u32(&full[s]), 0) : 0;
                        auto load = [&](uint8_t *d, const CUtensorMap *m, int c, int r, int plane) {
                            if constexpr (PAIR) tma_load_3d_pair(d, m, bar, c, r, plane);
                            else tma_load_3d(d, m, &full[s], c, r, plane);
                        };
                        if constexpr (AMN) {
#pragma unroll
                            for (int b = 0; b < kLanes / 64; ++b) load(da + b * 8192, &map_a, ia + 64 * b, at, pa);
                        } else {
                            load(da, &map_a, at, ia, pa);
                        }
                        if constexpr (BMN) {
                            for (int b = 0; b < cols / 64; ++b) load(db + b * 8192, &map_b, jb + 64 * b, at, pb);
                        } else {
                            load(db, &map_b, at, jb, pb);
                        }
                    }
                }
            }
        }
    } else if (warp == 1 && one && (!PAIR || rank == 0)) {
        // ---- products
        const uint32_t idesc = idesc_f16kind_f32(kTileLanes, bn, AMN, BMN, F8 ? kMmaE4M3 : kMmaBF16);
        const uint32_t at = smem_u32(sm);
        const uint64_t desc_a = AMN ? mnmajor_desc(at, 64, 0) : kmajor_desc(at, kLanes, 0),
                       desc_b = BMN ? mnmajor_desc(at + kABytes, 64, 0) : kmajor_desc(at + kABytes, cols, 0);
        auto commit = [&](uint64_t *bar) {
            if constexpr (PAIR) umma_commit_pair(bar);
            else umma_commit(bar);
        };
        int turn = 0;
        bool go = true;
        for (unsigned t = first; go && t < tiles; t += step)
            for (int c0 = b0; go && c0 < b1; c0 += a.chunk, ++turn) {
                const int acc = turn & 1, n = (min(b1, c0 + a.chunk) - c0) * a.npairs;
                if (!wait(&drained[acc], ((uint32_t)(turn >> 1) & 1u) ^ 1u)) {
                    fail = 1;
                    go = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tbase + acc * (tcols / 2);
                for (int k = 0; k < n; ++k, ring.step()) {
                    const int s = ring.s;
                    if (!wait(&full[s], ring.round & 1u)) {
                        fail = 1;
                        go = false;
                        break;
                    }
                    tc_fence_after();
                    // a stage and a step of 32 bytes of k further: 16-byte units in the low bits
                    const uint64_t sa = desc_a + (uint32_t)(s * stage) / 16, sb = desc_b + (uint32_t)(s * stage) / 16;
#pragma unroll
                    for (uint32_t q = 0; q < 4; ++q) {
                        const uint64_t da = sa + q * (AMN ? 128 : 2), db = sb + q * (BMN ? 128 : 2);
                        const uint32_t more = k > 0 || q > 0;
                        if constexpr (PAIR && F8) umma_f8_pair(d, da, db, idesc, more);
                        else if constexpr (PAIR) umma_bf16_pair(d, da, db, idesc, more);
                        else if constexpr (F8) umma_f8(d, da, db, idesc, more);
                        else umma_bf16(d, da, db, idesc, more);
                    }
                    commit(&empty[s]);
                }
                if (go) commit(&done[acc]);
            }
    } else if (!PROMOTE && warp >= 2 && a.staged && !a.out_f32) {
        // ---- epilogue through shared memory: this warp's 32 lanes, and every other 32 columns
        const uint32_t quad = warp & 3, half = (uint32_t)(warp - 2) >> 2, bar = 2 + half, row = lane >> 2;
        const bool leader = quad == 2 && one;   // warps 2 and 6
        uint8_t *const both = sm + stages * stage + half * 4 * kBuffer;
        // where a lane's row of a matrix lies: token lane % 8 (of 8), features 8 (lane / 8) on of this warp's
        const uint32_t chunk = (quad & 1) * 4 + (lane >> 3), at_row = (quad >> 1) * (kBuffer / 2) + (lane & 7) * 128 +
                                                                      ((chunk ^ (lane & 7)) << 4);
        int turn = 0, late = 0, used = 0;
        uint32_t loads = 0;   // parities of the loads into either pair of buffers
        // a pair of buffers is filled between two barriers: with 64 columns, or with z and y of 32
        const int width = EPI && a.z ? 32 : 64;
        for (unsigned t = first; t < tiles; t += step, ++turn) {
            const int acc = turn & 1;
            const Place p = place_of(t, mt, nt, kGroup);
            const int i0 = p.mi * kTileLanes + (PAIR ? rank * kLanes : 0), j0 = p.nj * bn;
            // the columns from c0 on of the residual, into the pair of buffers `to` (the leader)
            auto request = [&](int c0, int to) {
                if (c0 >= bn || j0 + c0 >= a.nj) return;
                const int slices = c0 + 32 < bn ? 2 : 1;
                uint64_t *arrived = &loaded[half * 2 + to];
                mbar_arrive_expect_tx(arrived, slices * kBuffer);
                for (int q = 0; q < slices; ++q) {
                    uint8_t *b = both + (to * 2 + q) * kBuffer;
                    tma_load_3d(b, &map_residual, arrived, i0, j0 + c0 + 32 * q, 0);
                    tma_load_3d(b + kBuffer / 2, &map_residual, arrived, i0 + 64, j0 + c0 + 32 * q, 0);
                }
            };
            // while the tile's products run, its residual: a half has two pairs of 64 columns at most (width is 64
            // here, as z and a residual together are not staged)
            if (EPI && a.residual && leader) {
                bulk_wait_read_all();
                request(half * width, used);
                request(half * width + 2 * width, used ^ 1);
            }
            float bias[4], si[4];
            if constexpr (EPI)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const long long i = i0 + (long long)(quad * 32 + 8 * g + row);
                    bias[g] = a.bias && i < a.ni ? __bfloat162float(((const __nv_bfloat16 *)a.bias)[i]) : 0.f;
                    if constexpr (F8) si[g] = i < a.ni ? a.scale_i[i] : 0.f;
                }
            // a wait that ran out ends no loop whose barriers other warps are in: what follows is not waited for
            if (!late && !wait(&done[acc], (uint32_t)(turn >> 1) & 1u)) fail = late = 1;
            tc_fence_after();
            const uint32_t from = tbase + (quad << 21) + acc * (tcols / 2);
#pragma unroll 1
            for (int c0 = half * width; c0 < bn && j0 + c0 < a.nj; c0 += 2 * width, used ^= 1) {
                uint8_t *buffers = both + used * 2 * kBuffer;
                const int slices = width == 64 && c0 + 32 < bn ? 2 : 1;
                // 8 KB for 32 columns from j on, as two boxes of 64 lanes
                auto store = [&](const CUtensorMap *m, uint8_t *b, int j) {
                    tma_store_3d(m, b, i0, j, 0);
                    tma_store_3d(m, b + kBuffer / 2, i0 + 64, j, 0);
                };
                if (leader && !(EPI && a.residual)) bulk_wait_read_but_one();   // what last left these buffers has been read
#pragma unroll 1
                for (int slice = 0; slice < slices; ++slice) {
                    const int c = c0 + 32 * slice;
                    const uint32_t to = smem_u32(buffers + slice * kBuffer) + at_row;
                    // v[r]: column 8 (r / 4 % 4) + 2 (lane % 4) + r % 2, feature 8 (2 (r / 16) + r / 2 % 2) + lane / 4
                    float v[32];
                    tmem_ld_frag32(from + c, v);
                    tmem_ld_frag32(from + (16u << 16) + c, v + 16);
                    tmem_ld_wait();
                    auto put32 = [&](uint32_t at) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const float *f = v + 16 * (g >> 1) + 4 * q + 2 * (g & 1);
                                w[g] = bf16x2_pack(f[0], f[1]);
                            }
                            stsm_x4_trans(at + q * 1024, w);
                        }
                    };
                    if constexpr (EPI) {
                        if constexpr (F8)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const long long col = j0 + (long long)c + 8 * q + 2 * (lane & 3) + e;
                                    const float sj = col < a.nj ? a.scale_j[col] : 0.f;
#pragma unroll
                                    for (int g = 0; g < 4; ++g) v[16 * (g >> 1) + 4 * q + 2 * (g & 1) + e] *= si[g] * sj;
                                }
                        if (a.bias)
#pragma unroll
                            for (int r = 0; r < 32; ++r) v[r] += bias[2 * (r / 16) + r / 2 % 2];
                    }
                    if (slice == 0 && !(EPI && a.residual)) named_sync(bar, kEpilogue / 2);   // the buffers are free
                    if constexpr (EPI) {
                        if (__builtin_expect(a.z != nullptr, 0)) put32(to + kBuffer);
                        activate<32>(v, a.activation);
                        if (__builtin_expect(a.residual != nullptr, 0)) {
                            if (slice == 0) {
                                if (!late && !wait(&loaded[half * 2 + used], loads >> used & 1u)) fail = late = 1;
                                loads ^= 1u << used;
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint32_t w[4];
                                ldsm_x4_trans(w, buffers + slice * kBuffer + at_row + q * 1024);
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    float f[2];
                                    bf16x2_widen(w[g], f);
                                    v[16 * (g >> 1) + 4 * q + 2 * (g & 1)] += f[0];
                                    v[16 * (g >> 1) + 4 * q + 2 * (g & 1) + 1] += f[1];
                                }
                            }
                        }
                    }
                    put32(to);
                }
                fence_proxy_async_smem();
                named_sync(bar, kEpilogue / 2);
                if (leader) {
                    store(&map_out, buffers, j0 + c0);
                    if (slices == 2) store(&map_out, buffers + kBuffer, j0 + c0 + 32);
                    if (EPI && a.z) store(&map_z, buffers + kBuffer, j0 + c0);
                    bulk_commit();
                }
            }
            drained_by(acc);
        }
        if (leader) bulk_wait_all();   // nothing is left in the buffers
    } else if (warp >= 2) {
        // ---- epilogue: this warp's 32 lanes and half of the columns, in units of 16
        const uint32_t quad = warp & 3, half = (uint32_t)(warp - 2) >> 2;
        const int per = half_columns(bn);
        uint8_t *const got = sm + stages * stage;   // split: [block][its columns of this block's share][lanes]
        // staged: [2][32 columns][lanes] for this half
        uint8_t *const both = sm + stages * stage + half * 4 * kBuffer;
        const uint32_t bar = 2 + half;
        const bool leader = quad == 2 && one;   // warps 2 and 6
        int turn = 0, used = 0, late = 0;
        uint32_t loads = 0;   // parities of the loads into either
        bool go = true;
        for (unsigned t = first; go && t < tiles; t += step) {
            const Place p = place_of(t, mt, nt, kGroup);
            const long long i = (long long)p.mi * kTileLanes + (PAIR ? rank * kLanes : 0) + quad * 32 + lane;
            int h0 = half * per, h = min(per, bn - h0), acc = 0;
            uint32_t row = 0;
            const int i0 = p.mi * kTileLanes + (PAIR ? rank * kLanes : 0);
            const int there = (int)min((long long)h, a.nj - ((long long)p.nj * bn + h0));   // staged: of this half
            auto request = [&](int c, int to) {   // columns c to c + 31 of the residual (the leader)
                if (c >= there) return;
                const int boxes = c + 16 < there ? 2 : 1;
                mbar_arrive_expect_tx(&loaded[half * 2 + to], boxes * kBuffer);
                for (int q = 0; q < boxes; ++q)
                    tma_load_3d(both + (to * 2 + q) * kBuffer, &map_residual, &loaded[half * 2 + to], i0,
                                p.nj * bn + h0 + c + 16 * q, 0);
            };
            if (EPI && a.staged && a.residual && leader) {   // the tile's first 64, while its products run
                bulk_wait_read_all();
                request(0, used);
                request(32, used ^ 1);
            }
            constexpr int kMostSums = PROMOTE ? (PAIR ? 128 : 64) : 16;   // of a half: bn is 256 or 128 at most
            float sum[kMostSums];
            if constexpr (PROMOTE)
#pragma unroll
                for (int c = 0; c < kMostSums; ++c) sum[c] = 0.f;
            for (int c0 = b0; c0 < b1; c0 += a.chunk, turn += PROMOTE) {
                acc = turn & 1;
                // a wait that ran out ends no loop whose barriers other warps are in
                if (!late && !wait(&done[acc], (uint32_t)(turn >> 1) & 1u)) {
                    fail = late = 1;
                    go = a.staged;
                }
                if (!go) break;
                tc_fence_after();
                row = tbase + (quad << 21) + acc * (tcols / 2) + h0;
                if constexpr (PROMOTE) {
#pragma unroll
                    for (int c = 0; c < kMostSums; c += 32)
                        if (c < h) {   // of 16 columns the second half is no sum, and not used (tensor_columns)
                            float v[32];
                            load_columns<32>(row + c, v);
#pragma unroll
                            for (int q = 0; q < 32; ++q) sum[c + q] += v[q];
                        }
                    drained_by(acc);
                }
            }
            // the first 16 sums; the others move up
            auto next = [&](int c) {
                if constexpr (PROMOTE) {
                    if (c > 0)
#pragma unroll
                        for (int q = 0; q < kMostSums - 16; ++q) sum[q] = sum[q + 16];
                } else {
                    load_columns<16>(row + c, sum);
                }
            };
            if (!PAIR && split > 1) {
                if (go) {
                    float *const part = (float *)sm + quad * 32 + lane;   // in the ring, whose stages are all free
#pragma unroll 1
                    for (int c = 0; c < h; c += 16) {
                        next(c);
#pragma unroll
                        for (int q = 0; q < 16; ++q) part[(h0 + c + q) * kLanes] = sum[q];
                    }
                }
                __syncwarp();
                cluster_wait();   // the other blocks have started
                fence_proxy_async_smem();
                named_sync(2, kEpilogue);
                const int share = bn / split, bytes = share * kLanes * 4;
                if (warp == 2 && one)
                    for (int to = 0; to < split; ++to)
                        bulk_copy_to_peer(mapa_shared(smem_u32(got + rank * bytes), to), sm + to * bytes, bytes,
                                          mapa_shared(smem_u32(&met), to));
                if (!wait(&met, 0)) fail = 1;
                __syncwarp();
                cluster_arrive_relaxed();   // nothing comes here any more
                per_half(share, half, h0, h);
            }
            const long long j = (long long)p.nj * bn + (!PAIR && split > 1 ? rank * (bn / split) : 0) + h0;
            if (go)
#pragma unroll 1
                for (int c = 0; c < h; c += 16) {
                    if (!PAIR && split > 1) {
                        const int share = bn / split;
                        const float *from = (const float *)got + (h0 + c) * kLanes + quad * 32 + lane;
#pragma unroll
                        for (int q = 0; q < 16; ++q) sum[q] = 0.f;
#pragma unroll 1
                        for (int b = 0; b < split; ++b, from += share * kLanes)
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                if (c + q < h) sum[q] += from[q * kLanes];
                    } else {
                        next(c);
                    }
                    const int valid = (int)min((long long)min(16, h - c), a.nj - j - c);
                    apply16<EPI, F8>(a, sum, i, j + c, valid);
                    if (!a.staged) {
                        store16<EPI>(a, sum, i, j + c, valid);
                        continue;
                    }
                    // fp32 results: 32 columns of a buffer, 16 at a time
                    float *mine = (float *)(both + used * 2 * kBuffer) + (c & 16) * kLanes + quad * 32 + lane;
                    if ((c & 16) == 0) {
                        if (EPI && a.residual) {
                            if (c < there) {
                                if (!late && !wait(&loaded[half * 2 + used], loads >> used & 1u)) fail = late = 1;
                                loads ^= 1u << used;
                            }
                        } else {
                            if (leader) bulk_wait_read_but_one();   // what last left this buffer has been read
                            named_sync(bar, kEpilogue / 2);
                        }
                    }
                    if (c < there) {   // behind the last column nothing was loaded, and the buffer may be in use
                        if (EPI && a.residual)
#pragma unroll
                            for (int q = 0; q < 16; ++q) sum[q] += mine[q * kLanes];
#pragma unroll
                        for (int q = 0; q < 16; ++q) mine[q * kLanes] = sum[q];
                    }
                    if ((c & 16) || c + 16 >= h) {
                        fence_proxy_async_smem();
                        named_sync(bar, kEpilogue / 2);
                        if (leader) {
                            const int c32 = c & ~31;
                            for (int q = c32; q <= c && q < there; q += 16)
                                tma_store_3d(&map_out, both + used * 2 * kBuffer + (q & 16) / 16 * kBuffer, i0,
                                             p.nj * bn + h0 + q, 0);
                            bulk_commit();
                            if (EPI && a.residual) {
                                bulk_wait_read_all();
                                request(c32 + 64, used);
                            }
                        }
                        used ^= 1;
                    }
                }
            if (!PROMOTE) {
                ++turn;
                drained_by(acc);
            }
        }
        if (leader) bulk_wait_all();   // nothing is left in the buffers
        if (!PAIR && split > 1) {
            __syncwarp();
            cluster_wait();   // nothing leaves from here any more: the others have all parts
        }
    }
    __syncwarp();
    if (!PAIR && split > 1 && warp < 2) {
        cluster_wait();
        cluster_arrive_relaxed();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (fail) {
        // what is under way ends before the memory it uses is given back (bounded)
        if (warp == 1 && one && (!PAIR || rank == 0)) {
            if constexpr (PAIR) umma_commit_pair(&drain);
            else umma_commit(&drain);
            wait(&drain, 0);
        }
        if (warp == 0 && one) {
            atomicOr(a.status, 1 << LDN_ERR_TIMEOUT);
            for (int s = 0; s < stages; ++s) {
                const uint32_t loads = ring.round + (s < ring.s);   // that went into stage s
                if (loads && (!PAIR || rank == 0)) wait(&full[s], (loads - 1) & 1u);
            }
        }
        __syncthreads();
    }
    if constexpr (PAIR) cluster_sync();   // neither block's barriers or memory are used any more
    if (warp == 1) {
        if constexpr (PAIR) tmem_dealloc_pair(tbase, tcols);
        else tmem_dealloc(tbase, tcols);
    }
}

}  // namespace linear
}  // namespace ldn
