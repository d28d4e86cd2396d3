// Linear layer with a fused epilogue, and its gradients, on tcgen05.
//
//   forward   z = x w^T + bias,  y = residual + alpha * act(z)
//   backward  dz = alpha * dy * act'(z);  dx = dz w;  dw = dz^T x;  dbias = sum_rows dz
//
// All three products are C[M][N] = sum_k A(m, k) B(n, k) with operands that
// are contiguous either along k (x, w in the forward pass; dz in dx) or along
// their own row index (w in dx; dz and x in dw). TMA brings both kinds into
// 128-byte-swizzled tiles, and the MMA's operand descriptors and major bits
// read either, so no transposed copy of anything is made.
//
// linear_gemm_kernel (320 threads): warp 0 TMA, warp 1 MMA issue, warps 2..9
// epilogue (two per TMEM lane quarter, half of the tile's columns each). Two
// shapes with the same 6 x 32 KB ring: CTA pairs with 256 x 256 tiles, and
// single CTAs with 128 x 128 tiles for problems with too few large tiles,
// with the sum over k split across CTAs when even those leave SMs idle
// (partial sums in the workspace, added in split order by
// linear_finish_kernel: no atomics, the same bits every run).
//
// Sums: the tensor core truncates as it accumulates, which costs a relative
// error of about 1.1e-9 per element of k (measured: 1.0e-5 at k = 9216, 2.3e-5
// at 20480, against 1e-6 for fp32 FMAs). So the accumulator is moved out of
// TMEM every 512 elements of k and added up in the epilogue warps' registers
// with rounding to nearest, while the tensor core fills the other of two
// accumulators; the epilogue warps are otherwise idle during the main loop.
#include "common.cuh"
#include "internal.h"

namespace klein {

namespace {

constexpr int kLinTile = 128 * 64 * 2;         // one operand tile: 128 rows (or columns) x 64 k, bf16
constexpr int kLinStage = 2 * kLinTile;        // A and B
constexpr int kLinStages = 6;
constexpr int kLinRing = kLinStages * kLinStage;
constexpr int kLinStaging = 8 * 4096;          // per epilogue warp: 32 rows x 32 fp32 columns
constexpr int kLinSmem = kLinRing + kLinStaging + 256 + 1024;
constexpr int kLinThreads = 320;
constexpr int kLinChunk = 8;                   // k blocks (of 64) per TMEM accumulation
constexpr int kLinPlanSms = 148;               // the B200's SM count: plans and workspace sizes do not depend on the device

// Shared-memory descriptor of an operand tile that is contiguous along its
// row index (MN-major), written by TMA in boxes of 64 rows x 64 k with
// 128-byte swizzling: lines of 64 row indices (128 B), 8 k per 1 KB atom
// (stride byte offset), the next 64 row indices one box later (leading byte
// offset).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t box_bytes) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(box_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ float lin_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(z); GELU in its tanh form, 0.5 z (1 + tanh u) = z / (1 + e^(-2u)).
__device__ __forceinline__ float lin_act(float z, int act) {
  if (act == kActSilu) return silu(z);
  if (act == kActGelu) return __fdividef(z, 1.0f + __expf(-kGelu2C * (z + kGeluA * z * z * z)));
  return z;
}

// act'(z). silu' = s + z s (1 - s); gelu' = s + z s (1 - s) d(2u)/dz with s = sigmoid(2u).
// Far out s (1 - s) is 0 while z or z^3 grows; the tails are taken apart so
// that 0 times an overflow cannot appear.
__device__ __forceinline__ float lin_act_grad(float z, int act) {
  if (act == kActNone) return 1.0f;
  if (fabsf(z) > 40.0f) return z > 0.f ? 1.0f : 0.0f;
  if (act == kActSilu) {
    const float s = lin_sigmoid(z);
    return s + z * s * (1.0f - s);
  }
  const float s = lin_sigmoid(kGelu2C * (z + kGeluA * z * z * z));
  return s + z * s * (1.0f - s) * kGelu2C * (1.0f + 3.0f * kGeluA * z * z);
}

__device__ __forceinline__ float lin_load(const void* p, long long i, int f32) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// The epilogue of up to four columns col..col+3 of one row (count valid
// ones): bias, saved pre-activation, activation, alpha, residual, output.
// The residual is read before the output is written, element by element, so
// the two may be the same matrix.
__device__ __forceinline__ void lin_finish4(const LinEpi& e, long long row, int col, float4 v, float4 bias) {
  float z[4] = {v.x + bias.x, v.y + bias.y, v.z + bias.z, v.w + bias.w};
  const int count = e.n - col < 4 ? e.n - col : 4;
  float r[4] = {0.f, 0.f, 0.f, 0.f};
  if (e.res) {
    const long long ri = row * e.res_ld + col;
    if (count == 4 && e.res_vec) {
      if (e.res_f32) {
        const float4 t = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.res) + ri);
        r[0] = t.x; r[1] = t.y; r[2] = t.z; r[3] = t.w;
      } else {
        const uint2 t = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(e.res) + ri);
        const float2 lo = unpack_bf16(t.x), hi = unpack_bf16(t.y);
        r[0] = lo.x; r[1] = lo.y; r[2] = hi.x; r[3] = hi.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) r[i] = lin_load(e.res, ri + i, e.res_f32);
    }
  }
  if (e.z) {  // the pre-activation is kept in bf16, as the layer's other activations are
    __nv_bfloat16* zp = e.z + row * e.z_ld + col;
    if (count == 4 && e.z_vec) {
      *reinterpret_cast<uint2*>(zp) = make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) zp[i] = __float2bfloat16_rn(z[i]);
    }
  }
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fmaf(e.alpha, lin_act(z[i], e.act), r[i]);
  const long long oi = row * e.out_ld + col;
  if (e.out_f32) {
    float* o = reinterpret_cast<float*>(e.out) + oi;
    if (count == 4 && e.out_vec) {
      *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) o[i] = y[i];
    }
  } else {
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(e.out) + oi;
    if (count == 4 && e.out_vec) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) o[i] = __float2bfloat16_rn(y[i]);
    }
  }
}

__device__ __forceinline__ float4 lin_bias4(const LinEpi& e, int col) {
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (e.bias) {
    if (col + 0 < e.n) b.x = __ldg(e.bias + col);
    if (col + 1 < e.n) b.y = __ldg(e.bias + col + 1);
    if (col + 2 < e.n) b.z = __ldg(e.bias + col + 2);
    if (col + 3 < e.n) b.w = __ldg(e.bias + col + 3);
  }
  return b;
}

}  // namespace

// One work item = (output tile, share of k): item i is tile i % tiles, split i / tiles.
template <bool AMN, bool BMN, bool PAIR>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const LinGemmArgs g) {
  constexpr int kTileM = PAIR ? 256 : 128, kTileN = kTileM;
  constexpr int kCols = kTileN / 2;  // accumulator columns per epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLinRing + kLinStaging);
  uint64_t* empty = full + kLinStages;
  uint64_t* acc_full = empty + kLinStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kLinStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], PAIR ? 512 : 256);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * kTileN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * kTileN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();  // operands and outputs are touched only after the previous kernel completes

  const int tiles = g.m_tiles * g.n_tiles;
  const int items = tiles * g.splits;
  const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int step = PAIR ? gridDim.x >> 1 : gridDim.x;
  constexpr uint32_t idesc =
      idesc_bf16_f32(kTileM, kTileN) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u);
  auto k_begin = [&](int split) { return static_cast<int>(static_cast<long long>(g.k_blocks) * split / g.splits); };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      StageLog log;
      bool ok = true;
      for (int item = first; ok && item < items; item += step) {
        const int tile = item % tiles, split = item / tiles;
        const int mi = g.n_fastest ? tile / g.n_tiles : tile % g.m_tiles;
        const int ni = g.n_fastest ? tile % g.n_tiles : tile / g.m_tiles;
        const int row = mi * kTileM + 128 * rank, col = ni * kTileN + 128 * rank;
        const int kb1 = k_begin(split + 1);
        for (int kb = k_begin(split); kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, 0x301)) { ok = false; break; }
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], PAIR ? 2 * kLinStage : kLinStage);
            log.armed(stage, phase);
          }
          uint8_t* sa = smem + stage * kLinStage;
          uint8_t* sb = sa + kLinTile;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int c0, int c1) {
            if (PAIR) tma_load_2d_pair(dst, map, mapa_shared(smem_u32(&full[stage]), 0), c0, c1);
            else tma_load_2d(dst, map, &full[stage], c0, c1);
          };
          if (AMN) {
            load(sa, &map_a, row, kb * 64);
            load(sa + kLinTile / 2, &map_a, row + 64, kb * 64);
          } else {
            load(sa, &map_a, kb * 64, row);
          }
          if (BMN) {
            load(sb, &map_b, col, kb * 64);
            load(sb + kLinTile / 2, &map_b, col + 64, kb * 64);
          } else {
            load(sb, &map_b, kb * 64, col);
          }
          if (++stage == kLinStages) { stage = 0; phase ^= 1; }
        }
      }
      // No TMA write of this CTA (or pair: the leader's barriers count both
      // CTAs' bytes, and the cluster barrier below keeps the other CTA alive)
      // may land after it exits.
      if (leader) log.drain(full, kLinStages, 0x305);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int chunk = 0;
      bool ok = true;
      for (int item = first; ok && item < items; item += step) {
        const int split = item / tiles;
        const int kb0 = k_begin(split), kb1 = k_begin(split + 1);
        for (int kb = kb0; kb < kb1; ++kb) {
          const int in_chunk = (kb - kb0) % kLinChunk;
          const int acc = chunk & 1;
          if (in_chunk == 0) {
            if (!mbar_wait(&acc_empty[acc], ((chunk >> 1) & 1) ^ 1, 0x302)) { ok = false; break; }
            tc_fence_after();
          }
          if (!mbar_wait(&full[stage], phase, 0x303)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * kTileN;
          const uint32_t a0 = smem_u32(smem + stage * kLinStage);
          const uint32_t b0 = a0 + kLinTile;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t da = AMN ? sw128_desc_mn(a0 + 2048 * k, kLinTile / 2) : sw128_desc(a0 + 32 * k);
            const uint64_t db = BMN ? sw128_desc_mn(b0 + 2048 * k, kLinTile / 2) : sw128_desc(b0 + 32 * k);
            if (PAIR) umma_bf16_pair(d, da, db, idesc, (in_chunk | k) != 0);
            else umma_bf16(d, da, db, idesc, (in_chunk | k) != 0);
          }
          if (PAIR) umma_commit_pair(&empty[stage], 0x3); else umma_commit(&empty[stage]);
          if (++stage == kLinStages) { stage = 0; phase ^= 1; }
          if (in_chunk == kLinChunk - 1 || kb == kb1 - 1) {
            if (PAIR) umma_commit_pair(&acc_full[acc], 0x3); else umma_commit(&acc_full[acc]);
            ++chunk;
          }
        }
      }
      // every MMA issued here has completed before TMEM is freed
      if (PAIR) umma_commit_pair(drain, 0x1); else umma_commit(drain);
      mbar_wait(drain, 0, 0x306);
    }
  } else {
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;  // which half of the tile's columns
    float* stg = reinterpret_cast<float*>(smem + kLinRing + (warp - 2) * 4096);
    const int sub = lane >> 3, c4 = lane & 7;  // after the transposition: row 4 i + sub, columns 4 c4..4 c4 + 3
    int chunk = 0;
    bool ok = true;
    for (int item = first; ok && item < items; item += step) {
      const int tile = item % tiles, split = item / tiles;
      const int mi = g.n_fastest ? tile / g.n_tiles : tile % g.m_tiles;
      const int ni = g.n_fastest ? tile % g.n_tiles : tile / g.m_tiles;
      const int chunks = (k_begin(split + 1) - k_begin(split) + kLinChunk - 1) / kLinChunk;
      float acc[kCols];
      for (int c = 0; c < chunks; ++c, ++chunk) {
        const int buf = chunk & 1;
        if (!mbar_wait(&acc_full[buf], (chunk >> 1) & 1, 0x304)) { ok = false; break; }
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + buf * kTileN + part * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
        if (c == 0) {
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) tmem_ld32(taddr + 32 * i, acc + 32 * i);
        } else {
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) {
            float v[32];
            tmem_ld32(taddr + 32 * i, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[32 * i + j] += v[j];
          }
        }
        tc_fence_before();
        if (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), 0));
        else mbar_arrive(&acc_empty[buf]);
      }
      if (!ok) break;
      // Each thread holds one row; through shared memory (16-byte chunks,
      // XOR-swizzled by row) a warp's 32 x 32 piece turns into whole row
      // segments, so that residual reads and output writes fill their sectors.
      const int row0 = mi * kTileM + 128 * rank + quarter * 32;
      const int col0 = ni * kTileN + part * kCols;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        if (row0 >= g.epi.m || col0 + 32 * i >= g.epi.n) break;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(stg + lane * 32 + ((j ^ (lane & 7)) << 2)) =
              make_float4(acc[32 * i + 4 * j], acc[32 * i + 4 * j + 1], acc[32 * i + 4 * j + 2], acc[32 * i + 4 * j + 3]);
        __syncwarp();
        const int col = col0 + 32 * i + 4 * c4;
        if (g.splits > 1) {
          float* p = g.partial + (static_cast<long long>(split) * g.epi.m + row0) * g.partial_ld + col;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int rr = 4 * r + sub;
            if (row0 + rr < g.epi.m)
              *reinterpret_cast<float4*>(p + rr * g.partial_ld) =
                  *reinterpret_cast<const float4*>(stg + rr * 32 + ((c4 ^ (rr & 7)) << 2));
          }
        } else if (col < g.epi.n) {
          const float4 bias = lin_bias4(g.epi, col);
#pragma unroll 4
          for (int r = 0; r < 8; ++r) {
            const int rr = 4 * r + sub;
            if (row0 + rr < g.epi.m)
              lin_finish4(g.epi, row0 + rr, col, *reinterpret_cast<const float4*>(stg + rr * 32 + ((c4 ^ (rr & 7)) << 2)),
                          bias);
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if (PAIR) cluster_sync(); else __syncthreads();  // every MMA and epilogue is done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, 2 * kTileN); else tmem_dealloc(tmem_base, 2 * kTileN);
  }
}

// Adds the splits' partial sums in split order and applies the epilogue.
__global__ void __launch_bounds__(256) linear_finish_kernel(const float* partial, long long partial_ld, int splits,
                                                            const LinEpi e) {
  pdl_trigger();
  pdl_wait();
  const int groups = (e.n + 3) / 4;
  const long long total = static_cast<long long>(e.m) * groups;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long row = i / groups;
    const int col = static_cast<int>(i - row * groups) * 4;
    const float* p = partial + row * partial_ld + col;
    float4 s = *reinterpret_cast<const float4*>(p);
    for (int k = 1; k < splits; ++k) {
      const float4 t = *reinterpret_cast<const float4*>(p + k * (e.m * partial_ld));
      s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
    }
    lin_finish4(e, row, col, s, lin_bias4(e, col));
  }
}

// Few rows (m <= MV <= 4): the weights are read once, straight into registers,
// WPO warps per output column (8 when there are too few columns to fill the
// GPU with one warp each), fp32 FMAs, one value per row and warp reduced by
// shuffles. Bound by the weights' bytes.
template <int MV, int WPO>
__global__ void __launch_bounds__(256) linear_rows_kernel(const __nv_bfloat16* x, long long x_ld,
                                                          const __nv_bfloat16* w, long long w_ld, int k,
                                                          const LinEpi e) {
  __shared__ float part[8][MV];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * (8 / WPO) + warp / WPO;
  float s[MV];
#pragma unroll
  for (int m = 0; m < MV; ++m) s[m] = 0.f;
  if (col < e.n) {
    const __nv_bfloat16* wr = w + static_cast<long long>(col) * w_ld;
    const int k8 = k & ~7;
    auto add8 = [&](uint4 wv, int at) {
      const float2 w0 = unpack_bf16(wv.x), w1 = unpack_bf16(wv.y), w2 = unpack_bf16(wv.z), w3 = unpack_bf16(wv.w);
#pragma unroll
      for (int m = 0; m < MV; ++m) {
        if (m < e.m) {
          const uint4 xv = *reinterpret_cast<const uint4*>(x + m * x_ld + at);
          const float2 x0 = unpack_bf16(xv.x), x1 = unpack_bf16(xv.y), x2 = unpack_bf16(xv.z), x3 = unpack_bf16(xv.w);
          s[m] = fmaf(w0.x, x0.x, fmaf(w0.y, x0.y, s[m]));
          s[m] = fmaf(w1.x, x1.x, fmaf(w1.y, x1.y, s[m]));
          s[m] = fmaf(w2.x, x2.x, fmaf(w2.y, x2.y, s[m]));
          s[m] = fmaf(w3.x, x3.x, fmaf(w3.y, x3.y, s[m]));
        }
      }
    };
    constexpr int kStep = WPO * 256;
    int at = (warp % WPO) * 256 + lane * 8;
    for (; at + 3 * kStep < k8; at += 4 * kStep) {
      uint4 wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) wv[u] = __ldg(reinterpret_cast<const uint4*>(wr + at + u * kStep));
#pragma unroll
      for (int u = 0; u < 4; ++u) add8(wv[u], at + u * kStep);
    }
    for (; at < k8; at += kStep) add8(__ldg(reinterpret_cast<const uint4*>(wr + at)), at);
    if (warp % WPO == 0 && k8 + lane < k) {  // the last k % 8 elements
      const float wv = __bfloat162float(wr[k8 + lane]);
#pragma unroll
      for (int m = 0; m < MV; ++m)
        if (m < e.m) s[m] = fmaf(wv, __bfloat162float(x[m * x_ld + k8 + lane]), s[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < MV; ++m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[m] += __shfl_xor_sync(0xffffffffu, s[m], o);
  }
  if (WPO > 1) {
    if (lane == 0) {
#pragma unroll
      for (int m = 0; m < MV; ++m) part[warp][m] = s[m];
    }
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int m = 0; m < MV; ++m) {
      s[m] = part[0][m];
#pragma unroll
      for (int i = 1; i < WPO; ++i) s[m] += part[i][m];
    }
  }
  float v = s[0];
#pragma unroll
  for (int m = 1; m < MV; ++m) v = lane == m ? s[m] : v;
  if (col < e.n && lane < MV && lane < e.m) {
    const float z = v + (e.bias ? __ldg(e.bias + col) : 0.f);
    const float r = e.res ? lin_load(e.res, lane * e.res_ld + col, e.res_f32) : 0.f;
    if (e.z) e.z[lane * e.z_ld + col] = __float2bfloat16_rn(z);
    const float y = fmaf(e.alpha, lin_act(z, e.act), r);
    if (e.out_f32) reinterpret_cast<float*>(e.out)[lane * e.out_ld + col] = y;
    else reinterpret_cast<__nv_bfloat16*>(e.out)[lane * e.out_ld + col] = __float2bfloat16_rn(y);
  }
}

// dz = alpha * dy * act'(z) in bf16 (the operand type of the two products
// after it) and, for dbias, the sum of each block's rows per column, from the
// fp32 dz before that rounding. A block takes 256 columns (8 per lane) and a
// slab of rows, its 8 warps every eighth row.
__global__ void __launch_bounds__(256) linear_dz_kernel(const LinDzArgs a) {
  __shared__ float sums[8][256];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 256 + lane * 8;
  const long long r0 = static_cast<long long>(blockIdx.y) * a.slab;
  const long long r1 = r0 + a.slab < a.m ? r0 + a.slab : a.m;
  const int count = a.n - col < 8 ? (a.n - col < 0 ? 0 : a.n - col) : 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (long long r = r0 + warp; r < r1; r += 8) {
    if (count <= 0) break;
    float d[8];
    const long long di = r * a.dout_ld + col;
    if (count == 8 && a.dout_vec) {
      if (a.dout_f32) {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.dout) + di);
        const float4 t0 = p[0], t1 = p[1];
        d[0] = t0.x; d[1] = t0.y; d[2] = t0.z; d[3] = t0.w;
        d[4] = t1.x; d[5] = t1.y; d[6] = t1.z; d[7] = t1.w;
      } else {
        const uint4 t = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.dout) + di);
        const float2 f0 = unpack_bf16(t.x), f1 = unpack_bf16(t.y), f2 = unpack_bf16(t.z), f3 = unpack_bf16(t.w);
        d[0] = f0.x; d[1] = f0.y; d[2] = f1.x; d[3] = f1.y;
        d[4] = f2.x; d[5] = f2.y; d[6] = f3.x; d[7] = f3.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = i < count ? lin_load(a.dout, di + i, a.dout_f32) : 0.f;
    }
    if (a.act != kActNone) {
      const __nv_bfloat16* zp = a.z + r * a.z_ld + col;
      float z[8];
      if (count == 8 && a.z_vec) {
        const uint4 t = *reinterpret_cast<const uint4*>(zp);
        const float2 f0 = unpack_bf16(t.x), f1 = unpack_bf16(t.y), f2 = unpack_bf16(t.z), f3 = unpack_bf16(t.w);
        z[0] = f0.x; z[1] = f0.y; z[2] = f1.x; z[3] = f1.y;
        z[4] = f2.x; z[5] = f2.y; z[6] = f3.x; z[7] = f3.y;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = i < count ? __bfloat162float(zp[i]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] *= lin_act_grad(z[i], a.act);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] *= a.alpha;
      s[i] += d[i];
    }
    if (a.dz)  // pitch a multiple of 8 columns: the padding columns get zeros
      *reinterpret_cast<uint4*>(a.dz + r * a.dz_ld + col) =
          make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
  }
  if (a.col_part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = s[i];
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < a.n) {
      float t = sums[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < 8; ++i) t += sums[i][threadIdx.x];
      a.col_part[static_cast<long long>(blockIdx.y) * a.n + c] = t;
    }
  }
}

// dbias[n] = sum of the slabs' column sums, in slab order.
__global__ void __launch_bounds__(256) linear_dbias_kernel(const float* part, int slabs, int n, float* dbias) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < slabs; ++i) s += part[static_cast<long long>(i) * n + c];
  dbias[c] = s;
}

// ------------------------------------------------------------------ host

// Tile shape and split count of one product from its sizes alone. The cost
// model counts tensor-core clocks of the busiest SM: a 64-deep step takes
// about 512 clocks for a pair's 256 x 256 tile and 300 for a single CTA's
// 128 x 128 (whose operand reads fill the shared-memory port), a tile's
// unoverlapped start and epilogue about 3000, and a split sum costs a second
// launch plus writing and reading the partial sums.
LinPlan plan_linear(long long m, long long n, long long k) {
  LinPlan best{};
  double best_cost = 0;
  const long long kb = (k + 63) / 64;
  for (int pair = 0; pair < 2; ++pair) {
    const long long t = pair ? 256 : 128;
    const long long tiles = ((m + t - 1) / t) * ((n + t - 1) / t);
    const long long slots = pair ? kLinPlanSms / 2 : kLinPlanSms;
    for (int s = 1; s <= (pair ? 4 : 16); ++s) {
      if (s > kb || (s > 1 && kb / s < 4)) break;
      const double waves = static_cast<double>((tiles * s + slots - 1) / slots);
      double cost = waves * (static_cast<double>((kb + s - 1) / s) * (pair ? 512 : 300) + 1000) + 2000;
      if (s > 1) cost += 5000 + 2.0 * s * m * ((n + 127) / 128 * 128) * 4 / 2500.0;
      if (best.splits == 0 || cost < best_cost) {
        best_cost = cost;
        best.pair = pair;
        best.splits = s;
      }
    }
  }
  best.partial_ld = (n + 127) / 128 * 128;
  best.partial_bytes = best.splits > 1 ? static_cast<size_t>(best.splits) * m * best.partial_ld * 4 : 0;
  return best;
}

template <bool AMN, bool BMN, bool PAIR>
static int launch_lin_one(const CUtensorMap& ma, const CUtensorMap& mb, const LinGemmArgs& g, cudaStream_t s) {
  static int slots_dev[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return -1;
  int& slots = slots_dev[dev];
  auto kernel = linear_gemm_kernel<AMN, BMN, PAIR>;
  if (slots == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem) != cudaSuccess) return -1;
    int n = num_sms();
    if (PAIR) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 * (n / 2));
      cfg.blockDim = dim3(kLinThreads);
      cfg.dynamicSmemBytes = kLinSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return -1;
    }
    slots = n;
  }
  const long long items = static_cast<long long>(g.m_tiles) * g.n_tiles * g.splits;
  const int groups = static_cast<int>(items < slots ? items : slots);
  const cudaError_t e = launch_kernel(kernel, dim3(PAIR ? 2 * groups : groups), dim3(kLinThreads), kLinSmem, s,
                                      PAIR ? 2 : 1, ma, mb, g);
  note_launch();
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

int launch_linear_gemm(const LinOperand& a, const LinOperand& b, int k, const LinEpi& epi, float* partial,
                       cudaStream_t s) {
  const LinPlan plan = plan_linear(epi.m, epi.n, k);
  const int tile = plan.pair ? 256 : 128;
  CUtensorMap ma, mb;
  auto encode = [&](CUtensorMap* map, const LinOperand& o, int rows) {
    // box: 64 k x 128 rows of a k-contiguous operand, 64 rows x 64 k of a row-contiguous one
    return o.mn_major ? make_map_2d(map, o.data, rows, k, static_cast<uint64_t>(o.ld) * 2, 64, 64)
                      : make_map_2d(map, o.data, k, rows, static_cast<uint64_t>(o.ld) * 2, 64, 128);
  };
  if (encode(&ma, a, epi.m) || encode(&mb, b, epi.n)) return -2;
  LinGemmArgs g{};
  g.m_tiles = (epi.m + tile - 1) / tile;
  g.n_tiles = (epi.n + tile - 1) / tile;
  g.k_blocks = (k + 63) / 64;
  g.splits = plan.splits;
  g.n_fastest = epi.n <= epi.m;  // the smaller operand stays in L2, the larger streams through once
  g.partial = partial;
  g.partial_ld = plan.partial_ld;
  g.epi = epi;
  int rc;
  if (!a.mn_major && !b.mn_major)
    rc = plan.pair ? launch_lin_one<false, false, true>(ma, mb, g, s) : launch_lin_one<false, false, false>(ma, mb, g, s);
  else if (!a.mn_major)
    rc = plan.pair ? launch_lin_one<false, true, true>(ma, mb, g, s) : launch_lin_one<false, true, false>(ma, mb, g, s);
  else
    rc = plan.pair ? launch_lin_one<true, true, true>(ma, mb, g, s) : launch_lin_one<true, true, false>(ma, mb, g, s);
  if (rc || plan.splits == 1) return rc;
  const long long quads = static_cast<long long>(epi.m) * ((epi.n + 3) / 4);
  const long long blocks = (quads + 255) / 256;
  const int grid = static_cast<int>(blocks < 8 * kLinPlanSms ? blocks : 8 * kLinPlanSms);
  const cudaError_t e = launch_kernel(linear_finish_kernel, dim3(grid), dim3(256), 0, s, 1,
                                      static_cast<const float*>(partial), g.partial_ld, plan.splits, epi);
  note_launch();
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

template <int MV>
static cudaError_t launch_rows_mv(const __nv_bfloat16* x, long long x_ld, const __nv_bfloat16* w, long long w_ld, int k,
                                  const LinEpi& e, cudaStream_t s) {
  if (e.n < 8 * kLinPlanSms && k >= 2048)  // one warp per column would leave most SMs with a few long serial rows
    return launch_kernel(linear_rows_kernel<MV, 8>, dim3(e.n), dim3(256), 0, s, 1, x, x_ld, w, w_ld, k, e);
  return launch_kernel(linear_rows_kernel<MV, 1>, dim3((e.n + 7) / 8), dim3(256), 0, s, 1, x, x_ld, w, w_ld, k, e);
}

int launch_linear_rows(const __nv_bfloat16* x, long long x_ld, const __nv_bfloat16* w, long long w_ld, int k,
                       const LinEpi& e, cudaStream_t s) {
  cudaError_t rc;
  if (e.m == 1) rc = launch_rows_mv<1>(x, x_ld, w, w_ld, k, e, s);
  else if (e.m == 2) rc = launch_rows_mv<2>(x, x_ld, w, w_ld, k, e, s);
  else rc = launch_rows_mv<4>(x, x_ld, w, w_ld, k, e, s);
  note_launch();
  return (rc == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

// Rows per block of linear_dz_kernel: about four blocks per SM, slabs a
// multiple of the 8 rows that a block's warps take at a time.
int lin_dz_slab(long long m, int n) {
  const long long col_blocks = (n + 255) / 256;
  long long slabs = (4 * kLinPlanSms + col_blocks - 1) / col_blocks;
  const long long most = (m + 31) / 32;
  if (slabs > most) slabs = most;
  if (slabs < 1) slabs = 1;
  const long long slab = (m + slabs - 1) / slabs;
  return static_cast<int>((slab + 7) / 8 * 8);
}

int launch_linear_dz(const LinDzArgs& a, float* dbias, cudaStream_t s) {
  const int slabs = static_cast<int>((a.m + a.slab - 1) / a.slab);
  cudaError_t e = launch_kernel(linear_dz_kernel, dim3((a.n + 255) / 256, slabs), dim3(256), 0, s, 1, a);
  note_launch();
  if (e == cudaSuccess && dbias) {
    e = launch_kernel(linear_dbias_kernel, dim3((a.n + 255) / 256), dim3(256), 0, s, 1,
                      static_cast<const float*>(a.col_part), slabs, a.n, dbias);
    note_launch();
  }
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

}  // namespace klein
