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
// linear_gemm_kernel: persistent CTA pairs, 256 x 256 output tiles, 5 x 32 KB
// ring, 384 threads: warp 0 TMA, warp 1 MMA issue, warps 4..11 epilogue (two
// per TMEM lane quarter, half of the tile's columns each), two TMEM accumulators so
// that a tile's epilogue overlaps the next one's main loop.
//
// Work is dealt out in whole tiles, one per pair and wave. The tiles of the last,
// partial wave are cut into equal parts along k when the plan finds that
// faster (few tiles, long k). Parts are dealt out part by part, so that the
// pairs at work read the same stretch of k of the operands; their sums go to
// the workspace, and linear_finish_kernel adds a tile's parts in the order of
// k and applies the epilogue. No atomics and no waiting between pairs: the
// same bits every run. (Shares of equal length that run across tiles balance
// a little better but spread over k: 1024 x 3072 x 20480, whose operands do
// not fit L2, took 124 us that way.)
//
// Sums: the tensor core truncates as it accumulates, which costs a relative
// error of about 1.1e-9 per element of k (measured: 1.0e-5 at k = 9216, 2.3e-5
// at 20480, against 1e-6 for fp32 FMAs). That is far below a bf16 output's
// rounding (2^-8), but not below an fp32 output's. So for fp32 outputs (FINE)
// the accumulator is moved out of TMEM every 512 elements of k and added up in
// the epilogue warps' registers with rounding to nearest, while the tensor
// core fills the other accumulator; these warps take registers over from the
// first four (3 x 168 = 72 + 2 x 216 per thread).
//
// An operand in two bf16 halves (dz and its remainders, for fp32 gradients) is
// multiplied in two passes over the same k, within every piece of work: first the
// high halves, then the low ones in chunks of their own. What is infinite in
// B is so in the first sum, with the right sign; the remainder's product with
// it (0 x inf, or an infinity of either sign) is left out.
#include "common.cuh"
#include "internal.h"

namespace klein {

namespace {

constexpr int kLinTile = 128 * 64 * 2;         // one operand tile: 128 rows (or columns) x 64 k, bf16
constexpr int kLinStage = 2 * kLinTile;        // A and B
constexpr int kLinStages = 5;
constexpr int kLinRing = kLinStages * kLinStage;
constexpr int kLinBox = 4096;                  // 32 rows of 128 bytes: 32 columns of fp32 or 64 of bf16
constexpr int kLinStaging = 8 * 2 * kLinBox;   // two per epilogue warp
constexpr int kLinBias = 8 * 128;              // 32 columns' bias per epilogue warp
constexpr int kLinSmem = kLinRing + kLinStaging + kLinBias + 256 + 1024;
static_assert(kLinSmem <= 227 * 1024, "shared memory of one CTA");
constexpr int kLinThreads = 384;
constexpr int kLinChunk = 8;                   // FINE: k blocks (of 64) per TMEM accumulation
constexpr int kLinSms = 148;                   // the B200's SM count: plans and workspace sizes do not depend on the device
constexpr int kLinPairs = kLinSms / 2;

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
// s and s - s^2 keep their relative precision down to an exponent of -87, where
// e^87 is the last denominator below 2^126 (s is 0 past it). At |z| = 100 both
// derivatives are 0 or 1, and z is taken there from then on: further out z^3 or
// an infinite z would meet that 0 (a NaN stays).
template <int ACT>
__device__ __forceinline__ float lin_act_grad(float z) {
  if (ACT == kActNone) return 1.0f;
  z = fabsf(z) > 100.0f ? copysignf(100.0f, z) : z;
  const float z2 = z * z;
  const float s = lin_sigmoid(ACT == kActSilu ? z : kGelu2C * z * fmaf(kGeluA, z2, 1.0f));
  const float t = z * (s - s * s);
  return ACT == kActSilu ? s + t : fmaf(t, kGelu2C * fmaf(3.0f * kGeluA, z2, 1.0f), s);
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
    if (col + 0 < e.n) b.x = e.bias[col];
    if (col + 1 < e.n) b.y = e.bias[col + 1];
    if (col + 2 < e.n) b.z = e.bias[col + 2];
    if (col + 3 < e.n) b.w = e.bias[col + 3];
  }
  return b;
}

}  // namespace

// A pair's share of the work: for w < waves the whole tile w * pairs + pair,
// then every pairs-th of the cut tiles' parts.
struct LinPiece {
  int mi, ni, kb0, kb1;
  int slot;  // where its sums go in the workspace, or -1: a whole tile, finished here
};

__device__ __forceinline__ void lin_tile(const LinGemmArgs& g, int tile, int& mi, int& ni) {
  mi = g.n_fastest ? tile / g.n_tiles : tile % g.m_tiles;
  ni = g.n_fastest ? tile % g.n_tiles : tile / g.m_tiles;
}

__device__ __forceinline__ bool lin_piece(const LinGemmArgs& g, int pair, int i, LinPiece& p) {
  if (i < g.waves) {
    const int tile = i * g.pairs + pair;
    if (tile >= g.whole) return false;
    lin_tile(g, tile, p.mi, p.ni);
    p.kb0 = 0;
    p.kb1 = g.k_blocks;
    p.slot = -1;
    return true;
  }
  const int item = (i - g.waves) * g.pairs + pair;
  if (item >= g.cut * g.parts) return false;
  const int part = item / g.cut;
  lin_tile(g, g.whole + item % g.cut, p.mi, p.ni);
  p.kb0 = static_cast<int>(static_cast<long long>(g.k_blocks) * part / g.parts);
  p.kb1 = static_cast<int>(static_cast<long long>(g.k_blocks) * (part + 1) / g.parts);
  p.slot = item;
  return true;
}

// ---- the epilogue's boxes: 32 rows of 128 bytes in shared memory, one row per
// lane, 16-byte pieces swizzled the way TMA does it (by row % 8), so that neither
// a lane's own row nor whole rows conflict.

__device__ __forceinline__ uint8_t* lin_piece16(uint8_t* box, int row, int i) {
  return box + row * 128 + ((i ^ (row & 7)) << 4);
}

// 32 columns of one row: all of a box of fp32, or half (0, 1) of one of bf16.
__device__ __forceinline__ void lin_box_write(uint8_t* box, int row, const float* v, bool f32, int half) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(lin_piece16(box, row, i)) =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(lin_piece16(box, row, 4 * half + i)) =
          make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  }
}

// v += those columns
__device__ __forceinline__ void lin_box_add(uint8_t* box, int row, float* v, bool f32, int half) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(lin_piece16(box, row, i));
      v[4 * i] += t.x;
      v[4 * i + 1] += t.y;
      v[4 * i + 2] += t.z;
      v[4 * i + 3] += t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 t = *reinterpret_cast<const uint4*>(lin_piece16(box, row, 4 * half + i));
      const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_bf16(u[j]);
        v[8 * i + 2 * j] += f.x;
        v[8 * i + 2 * j + 1] += f.y;
      }
    }
  }
}

__device__ __forceinline__ void lin_bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// until the bulk stores of this thread have read their shared memory / are done
__device__ __forceinline__ void lin_bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void lin_bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void lin_store_box(const CUtensorMap* map, const void* box, int col, int row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(box)), "r"(col), "r"(row)
               : "memory");
}

__device__ __forceinline__ void lin_store_raw(void* dst, const void* box, int bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(box)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void lin_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The epilogue element by element: this lane's column of a box of fp32 sums,
// 32 rows from row0 on. Any pitch, width and alignment; a row's 32 elements
// are one access of the warp. BATCH rows' residuals are in flight at a time
// (4608 x 9218 x 16 in batches of 8 and of 32: 89 and 43 us, with a residual 277 and 187).
template <bool OUT32, bool FULL, int BATCH>
__device__ __forceinline__ void lin_finish_column(const LinEpi& e, const uint8_t* box, int lane, int row0, int col) {
  const int rows = e.m - row0 < 32 ? e.m - row0 : 32;
  if (col >= e.n) return;
  const float bias = FULL && e.bias ? e.bias[col] : 0.f;
  const long long out_ld = e.out_ld, res_ld = e.res_ld, z_ld = e.z_ld;
  float* o32 = static_cast<float*>(e.out) + row0 * out_ld + col;
  __nv_bfloat16* o16 = static_cast<__nv_bfloat16*>(e.out) + row0 * out_ld + col;
  const float* r32 = static_cast<const float*>(e.res) + row0 * res_ld + col;
  const __nv_bfloat16* r16 = static_cast<const __nv_bfloat16*>(e.res) + row0 * res_ld + col;
  __nv_bfloat16* z16 = e.z + row0 * z_ld + col;
  const bool has_res = e.res != nullptr, res_f32 = e.res_f32, has_z = FULL && e.z != nullptr;
  const float alpha = e.alpha;
  const int act = FULL ? e.act : kActNone;
  const uint8_t* src = box + (lane & 3) * 4;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += BATCH) {
    float z[BATCH], res[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      z[i] = *reinterpret_cast<const float*>(src + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4)) + bias;
      res[i] = 0.f;
    }
    if (has_res) {
      if (res_f32) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (r0 + i < rows) res[i] = r32[i * res_ld];
      } else {
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (r0 + i < rows) res[i] = __bfloat162float(r16[i * res_ld]);
      }
      r32 += BATCH * res_ld;
      r16 += BATCH * res_ld;
    }
    if (has_z) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (r0 + i < rows) z16[i * z_ld] = __float2bfloat16_rn(z[i]);
      z16 += BATCH * z_ld;
    }
    if (act != kActNone) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) z[i] = lin_act(z[i], act);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const float y = fmaf(alpha, z[i], res[i]);
      if (r0 + i < rows) {
        if (OUT32) o32[i * out_ld] = y;
        else o16[i * out_ld] = __float2bfloat16_rn(y);
      }
    }
    o32 += BATCH * out_ld;
    o16 += BATCH * out_ld;
  }
}

// FINE: the output is fp32. FULL: the epilogue may have a bias, a saved
// pre-activation and an activation (the products of the backward pass never do).
template <bool AMN, bool BMN, bool FINE, bool FULL>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_res,
                       const LinGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLinRing + kLinStaging + kLinBias);
  uint64_t* empty = full + kLinStages;
  uint64_t* acc_full = empty + kLinStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* res_full = drain + 1;  // [8 epilogue warps]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kLinStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);  // one arrival per epilogue warp of the pair
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&res_full[i], 1);
    fence_barrier_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
    if (g.epi.tma) {
      tma_prefetch_desc(&map_out);
      if (g.epi.res) tma_prefetch_desc(&map_res);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barrier initialisation and the TMEM allocation are visible pair-wide
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();  // operands and outputs are touched only after the previous kernel completes

  const int pair0 = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  constexpr uint32_t idesc = idesc_bf16_f32(256, 256) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u);
  LinPiece p;

  // Loads here and below are plain ones, not __ldg: this kernel may start while
  // the one that writes an operand still runs (programmatic dependent launch),
  // and only plain loads see its writes after pdl_wait.
  if (warp < 4) {
    if (FINE) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        StageLog log;
        bool ok = true;
        for (int pair = pair0; ok && pair < g.pairs; pair += pairs) {
          for (int i = 0; ok && lin_piece(g, pair, i, p); ++i) {
            const int row = p.mi * 256 + 128 * rank, col = p.ni * 256 + 128 * rank;
            const int len = p.kb1 - p.kb0, steps = g.a_low ? 2 * len : len;
            for (int j = 0; j < steps; ++j) {
              if (!mbar_wait(&empty[stage], phase ^ 1, 0x301)) { ok = false; break; }
              if (leader) {
                mbar_arrive_expect_tx(&full[stage], 2 * kLinStage);
                log.armed(stage, phase);
              }
              uint8_t* sa = smem + stage * kLinStage;
              uint8_t* sb = sa + kLinTile;
              const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
              // the second pass over the piece's k reads A's low halves against the same B
              const int low = j < len ? 0 : g.a_low;
              const int k = (p.kb0 + (j < len ? j : j - len)) * 64;
              if (AMN) {
                tma_load_2d_pair(sa, &map_a, bar, row + low, k);
                tma_load_2d_pair(sa + kLinTile / 2, &map_a, bar, row + low + 64, k);
              } else {
                tma_load_2d_pair(sa, &map_a, bar, k + low, row);
              }
              if (BMN) {
                tma_load_2d_pair(sb, &map_b, bar, col, k);
                tma_load_2d_pair(sb + kLinTile / 2, &map_b, bar, col + 64, k);
              } else {
                tma_load_2d_pair(sb, &map_b, bar, k, col);
              }
              if (++stage == kLinStages) { stage = 0; phase ^= 1; }
            }
          }
        }
        // No TMA write of the pair may land after it exits: the leader's
        // barriers count both CTAs' bytes, and the cluster barrier below keeps
        // the other CTA alive.
        if (leader) log.drain(full, kLinStages, 0x305);
      }
    } else if (warp == 1) {
      if (lane == 0 && leader) {
        int stage = 0;
        uint32_t phase = 0;
        int chunk = 0;
        bool ok = true;
        for (int pair = pair0; ok && pair < g.pairs; pair += pairs) {
          for (int i = 0; ok && lin_piece(g, pair, i, p); ++i) {
            const int len = p.kb1 - p.kb0, steps = g.a_low ? 2 * len : len;
            for (int j = 0; ok && j < steps; ++chunk) {
              const int acc = chunk & 1;
              if (!mbar_wait(&acc_empty[acc], ((chunk >> 1) & 1) ^ 1, 0x302)) { ok = false; break; }
              tc_fence_after();
              const uint32_t d = tmem_base + acc * 256;
              const int first = j;
              int end = j < len ? len : steps;  // no chunk holds steps of both passes
              if (FINE && j + kLinChunk < end) end = j + kLinChunk;
              for (; j < end; ++j) {
                if (!mbar_wait(&full[stage], phase, 0x303)) { ok = false; break; }
                tc_fence_after();
                const uint32_t a0 = smem_u32(smem + stage * kLinStage);
                const uint32_t b0 = a0 + kLinTile;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint64_t da = AMN ? sw128_desc_mn(a0 + 2048 * k, kLinTile / 2) : sw128_desc(a0 + 32 * k);
                  const uint64_t db = BMN ? sw128_desc_mn(b0 + 2048 * k, kLinTile / 2) : sw128_desc(b0 + 32 * k);
                  umma_bf16_pair(d, da, db, idesc, j != first || k != 0);
                }
                umma_commit_pair(&empty[stage], 0x3);
                if (++stage == kLinStages) { stage = 0; phase ^= 1; }
              }
              if (ok) umma_commit_pair(&acc_full[acc], 0x3);
            }
          }
        }
        // every MMA issued here has completed before TMEM is freed
        umma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, 0x306);
      }
    }
  } else {
    if (FINE) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3;
    const int part = (warp - 4) >> 2;  // which half of the tile's columns
    const LinEpi& e = g.epi;
    uint8_t* boxes = smem + kLinRing + (warp - 4) * 2 * kLinBox;
    float* bias_row = reinterpret_cast<float*>(smem + kLinRing + kLinStaging + (warp - 4) * 128);
    uint64_t* rbar = res_full + (warp - 4);
    // What the epilogue asks of its arguments again and again, asked once.
    const bool tma = e.tma, has_bias = FULL && e.bias != nullptr, has_z = FULL && e.z != nullptr;
    const bool load_res = tma && e.res, res32 = e.res_f32;
    const int act = FULL ? e.act : kActNone;
    const float alpha = e.alpha;
    const int m = e.m, n = e.n;
    // A round is what the two boxes hold: 128 columns if everything is bf16, else 64.
    const bool wide = !FINE && !(load_res && res32);
    uint32_t res_phase = 0;  // parity of the next residual
    bool res_due = false;    // lane 0: a residual is on its way
    int chunk = 0;
    bool ok = true;
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_tmem(mapa_shared(smem_u32(&acc_empty[buf]), 0));
    };
    auto fetch_res = [&](int row0, int col) {  // lane 0: a round's residual, into boxes that nothing uses
      lin_bulk_wait_read();
      const int per_box = res32 ? 32 : 64;
      const bool two = (wide || res32) && col + per_box < n;
      mbar_arrive_expect_tx(rbar, two ? 2 * kLinBox : kLinBox);
      res_due = true;
      // (64 columns of bf16 lie in the second box if the output is fp32: the lane reads them all before it writes)
      tma_load_2d(boxes + (FINE && !res32 ? kLinBox : 0), &map_res, rbar, col, row0);
      if (two) tma_load_2d(boxes + kLinBox, &map_res, rbar, col + per_box, row0);
    };
    auto boxes_free = [&]() {
      if (lane == 0) lin_bulk_wait_read();
      __syncwarp();
    };
    // The boxes as they stand become columns col..col + cols - 1 of the output.
    auto store_boxes = [&](int cols, int row0, int col) {
      constexpr int per_box = FINE ? 32 : 64;
      lin_fence_async();
      __syncwarp();
      if (lane == 0) {
        lin_store_box(&map_out, boxes, col, row0);
        if (cols > per_box && col + per_box < n) lin_store_box(&map_out, boxes + kLinBox, col + per_box, row0);
        lin_bulk_commit();
      }
    };
    // 32 columns (the h-th 32 of the tile half at col0); v: this lane's row;
    // last: no more columns in the matrix.
    auto finish = [&](float* v, int h, int row0, int col0, bool last) {
      const int col = col0 + 32 * h;
      const int odd = h & 1;
      if (p.slot >= 0) {  // a part's sums, as the boxes are
        if (!odd) boxes_free();
        lin_box_write(boxes + odd * kLinBox, lane, v, true, 0);
        if (odd || last) {
          lin_fence_async();
          __syncwarp();
          if (lane == 0) {
            const int rb = 4 * rank + quarter, cb = 4 * part + h - odd;
            lin_store_raw(g.partial + ((static_cast<long long>(p.slot) * g.part_rb + rb) * g.part_cb + cb) * (kLinBox / 4),
                          boxes, odd ? 2 * kLinBox : kLinBox);
            lin_bulk_commit();
          }
        }
        return;
      }
      if (!tma) {  // pitches, widths or addresses that TMA cannot take: a column to a lane, row by row
        boxes_free();
        lin_box_write(boxes, lane, v, true, 0);
        __syncwarp();
        lin_finish_column<FINE, FULL, FINE ? 8 : 32>(e, boxes, lane, row0, col + lane);
        return;
      }
      if (has_bias) {
        __syncwarp();
        bias_row[lane] = col + lane < n ? e.bias[col + lane] : 0.f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 t = *reinterpret_cast<const float4*>(bias_row + i);
          v[i] += t.x;
          v[i + 1] += t.y;
          v[i + 2] += t.z;
          v[i + 3] += t.w;
        }
      }
      if (has_z && row0 + lane < m) {  // whole sectors of this lane's row
        __nv_bfloat16* zp = e.z + (row0 + lane) * e.z_ld + col;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          if (col + i < n)
            *reinterpret_cast<uint4*>(zp + i) = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                                                           pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
      }
      if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = lin_act(v[i], kActSilu);
      } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = lin_act(v[i], kActGelu);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= alpha;
      const int before = wide ? 32 * h : 32 * odd;  // columns of the round already in the boxes
      if (load_res) {
        if (before == 0) {
          if (!mbar_wait_warp(rbar, res_phase, 0x307)) { ok = false; return; }
          res_phase ^= 1;
          res_due = false;
        }
        lin_box_add(boxes + (res32 ? odd : (FINE ? 1 : h >> 1)) * kLinBox, lane, v, res32, odd);
      } else if (before == 0) {
        boxes_free();
      }
      lin_box_write(boxes + (FINE ? odd : (wide ? h >> 1 : 0)) * kLinBox, lane, v, FINE, odd);
      if (last || (!wide && odd)) {
        store_boxes(before + 32, row0, col - before);
        if (load_res && !last && lane == 0) fetch_res(row0, col + 32);
      }
    };
    for (int pair = pair0; ok && pair < g.pairs; pair += pairs) {
      for (int i = 0; ok && lin_piece(g, pair, i, p); ++i) {
        const int row0 = p.mi * 256 + 128 * rank + quarter * 32;
        const int col0 = p.ni * 256 + part * 128;
        int pieces = row0 < m && col0 < n ? (n - col0 + 31) / 32 : 0;  // of 32 columns, in the matrix
        if (pieces > 4) pieces = 4;
        if (load_res && p.slot < 0 && lane == 0 && pieces > 0) fetch_res(row0, col0);  // under the main loop
        if (FINE) {
          const int high = (p.kb1 - p.kb0 + kLinChunk - 1) / kLinChunk;
          const int chunks = g.a_low ? 2 * high : high;
          float acc[128];
          for (int c = 0; c < chunks; ++c, ++chunk) {
            const int buf = chunk & 1;
            if (!mbar_wait_warp(&acc_full[buf], (chunk >> 1) & 1, 0x304)) { ok = false; break; }
            tc_fence_after();
            const uint32_t taddr =
                tmem_base + buf * 256 + part * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (c == 0) {
                tmem_ld32(taddr + 32 * j, acc + 32 * j);
              } else {
                float v[32];
                tmem_ld32(taddr + 32 * j, v);
                if (FULL || c < high) {
#pragma unroll
                  for (int q = 0; q < 32; ++q) acc[32 * j + q] += v[q];
                } else {  // the low halves: nothing to a sum that B has made infinite or NaN
#pragma unroll
                  for (int q = 0; q < 32; ++q) acc[32 * j + q] += fabsf(acc[32 * j + q]) < INFINITY ? v[q] : 0.f;
                }
              }
            }
            release(buf);
          }
#pragma unroll 1
          for (int h = 0; ok && h < pieces; ++h) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float lo = h & 1 ? acc[32 + j] : acc[j], hi = h & 1 ? acc[96 + j] : acc[64 + j];
              v[j] = h & 2 ? hi : lo;
            }
            finish(v, h, row0, col0, h == pieces - 1);
          }
        } else {
          const int buf = chunk & 1;
          if (!mbar_wait_warp(&acc_full[buf], (chunk >> 1) & 1, 0x304)) { ok = false; break; }
          ++chunk;
          tc_fence_after();
          const uint32_t taddr = tmem_base + buf * 256 + part * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
          for (int h = 0; ok && h < pieces; ++h) {
            float v[32];
            tmem_ld32(taddr + 32 * h, v);
            if (h == pieces - 1) release(buf);
            finish(v, h, row0, col0, h == pieces - 1);
          }
          if (pieces == 0) release(buf);
        }
      }
    }
    if (lane == 0) {
      // when the CTA exits no store may still read shared memory, and (after a
      // wait that gave up) no residual may still be on its way
      lin_bulk_wait_all();
      if (res_due) mbar_wait(rbar, res_phase, 0x308);
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();  // every MMA and every epilogue of both CTAs is done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// The cut tiles: adds the parts' sums in the order of k and applies the
// epilogue. One block takes one 32 x 32 box of a tile, a float4 per thread.
__global__ void __launch_bounds__(256) linear_finish_kernel(const LinGemmArgs g) {
  pdl_trigger();
  pdl_wait();
  int mi, ni;
  lin_tile(g, g.whole + blockIdx.y, mi, ni);
  const int rb = blockIdx.x / g.part_cb, cb = blockIdx.x % g.part_cb;
  const int r = threadIdx.x >> 3, c4 = threadIdx.x & 7;
  const long long row = static_cast<long long>(mi) * 256 + rb * 32 + r;
  const int col = ni * 256 + cb * 32 + c4 * 4;
  if (row >= g.epi.m || col >= g.epi.n) return;
  const long long plane = static_cast<long long>(g.part_rb) * g.part_cb * (kLinBox / 4);
  const float* src = g.partial + blockIdx.y * plane + static_cast<long long>(blockIdx.x) * (kLinBox / 4) + r * 32 +
                     ((c4 ^ (r & 7)) << 2);
  float4 v = __ldcg(reinterpret_cast<const float4*>(src));
#pragma unroll 4
  for (int q = 1; q < g.parts; ++q) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(src + q * g.cut * plane));
    v.x += t.x;
    v.y += t.y;
    v.z += t.z;
    v.w += t.w;
  }
  lin_finish4(g.epi, row, col, v, lin_bias4(g.epi, col));
}

// Eight bf16 of a row from column k on, zeros past the row's end.
__device__ __forceinline__ uint4 lin_load8(const __nv_bfloat16* row, int k, int k_end) {
  if (k + 8 <= k_end) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t u[4] = {0u, 0u, 0u, 0u};
  const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < k_end) u[i >> 1] |= static_cast<uint32_t>(r[k + i]) << (16 * (i & 1));
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void lin_mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Few rows, or little of everything: the weights' bytes are all that counts,
// and they go straight from memory into registers. A block takes 8 NB rows of
// x and 16 columns (rows of w),
// its WARPS warps every WARPS-th stretch of 128 of k (16 warps for long rows of
// which there are too few to fill the SMs, else 8). Per 32 of k a lane loads 16
// bytes of two weight rows and of one row of x per NB: with lane = 4 g + t,
// row g (and g + 8) and k = 8 t .. 8 t + 7. Which elements of k a product step
// pairs is free as long as both operands agree, so those registers are the
// operands of two 16 x 8 x 16 warp-level products as they are, with weights as
// A and rows of x as B. (The 5th generation's products want both operands
// in shared memory and 128 rows; here the arithmetic is 1 % of the time.) The
// warps' sums are added in shared memory in a fixed order; like the large
// products they are moved to fp32 registers every 512 of k.
template <int NB, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) linear_rows_kernel(const __nv_bfloat16* x, long long x_ld,
                                                          const __nv_bfloat16* w, long long w_ld, int k,
                                                          const LinEpi e) {
  __shared__ float part[WARPS][8 * NB][17];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int col0 = blockIdx.x * 16;
  const int row0 = blockIdx.y * 8 * NB, rows = e.m - row0;
  // (rows past the last are read again, and not stored)
  const __nv_bfloat16* w0 = w + static_cast<long long>(col0 + g < e.n ? col0 + g : e.n - 1) * w_ld;
  const __nv_bfloat16* w1 = w + static_cast<long long>(col0 + g + 8 < e.n ? col0 + g + 8 : e.n - 1) * w_ld;
  const __nv_bfloat16* xr[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) xr[b] = x + static_cast<long long>(row0 + (8 * b + g < rows ? 8 * b + g : rows - 1)) * x_ld;
  float sum[NB][4], c[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[b][i] = c[b][i] = 0.f;
  auto step = [&](uint4 a, uint4 a8, const uint4* xv) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      lin_mma16816(c[b], a.x, a8.x, a.y, a8.y, xv[b].x, xv[b].y);
      lin_mma16816(c[b], a.z, a8.z, a.w, a8.w, xv[b].z, xv[b].w);
    }
  };
  int since = 0;
  for (int k0 = warp * 128; k0 < k; k0 += 128 * WARPS) {
    if (k0 + 128 <= k) {
      uint4 a[4], a8[4], xv[4][NB];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = k0 + 32 * u + 8 * t;
        a[u] = __ldcs(reinterpret_cast<const uint4*>(w0 + at));
        a8[u] = __ldcs(reinterpret_cast<const uint4*>(w1 + at));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b) xv[u][b] = *reinterpret_cast<const uint4*>(xr[b] + k0 + 32 * u + 8 * t);
#pragma unroll
      for (int u = 0; u < 4; ++u) step(a[u], a8[u], xv[u]);
    } else {
      for (int at = k0 + 8 * t; at - 8 * t < k; at += 32) {
        uint4 xv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) xv[b] = lin_load8(xr[b], at, k);
        step(lin_load8(w0, at, k), lin_load8(w1, at, k), xv);
      }
    }
    if (++since == 4) {
      since = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[b][i] += c[b][i];
          c[b][i] = 0.f;
        }
    }
  }
  // element (column g or g + 8 of w's 16, row 2 t or 2 t + 1 of x's 8)
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    part[warp][8 * b + 2 * t][g] = sum[b][0] + c[b][0];
    part[warp][8 * b + 2 * t + 1][g] = sum[b][1] + c[b][1];
    part[warp][8 * b + 2 * t][g + 8] = sum[b][2] + c[b][2];
    part[warp][8 * b + 2 * t + 1][g + 8] = sum[b][3] + c[b][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 128 * NB; i += 32 * WARPS) {
    const int r = i >> 4, col = col0 + (i & 15);
    if (r >= rows || col >= e.n) continue;
    float v = part[0][r][i & 15];
#pragma unroll
    for (int q = 1; q < WARPS; ++q) v += part[q][r][i & 15];
    const long long row = row0 + r;
    const float z = v + (e.bias ? e.bias[col] : 0.f);
    const float res = e.res ? lin_load(e.res, row * e.res_ld + col, e.res_f32) : 0.f;
    if (e.z) e.z[row * e.z_ld + col] = __float2bfloat16_rn(z);
    const float y = fmaf(e.alpha, lin_act(z, e.act), res);
    if (e.out_f32) static_cast<float*>(e.out)[row * e.out_ld + col] = y;
    else static_cast<__nv_bfloat16*>(e.out)[row * e.out_ld + col] = __float2bfloat16_rn(y);
  }
}

// dz = alpha * dy * act'(z) in bf16 (the operand type of the two products
// after it), with `low` also the bf16 remainder (the two together keep 16 bits
// of mantissa, for products whose output is fp32), and, for dbias, the sum of each block's rows per column, from the
// fp32 dz before that rounding. A block takes 256 columns (8 per lane) and a
// slab of rows, its 8 warps every eighth row.
template <int ACT>
__global__ void __launch_bounds__(256, 2) linear_dz_kernel(const LinDzArgs a) {
  __shared__ float sums[8][256];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 256 + lane * 8;
  const long long r0 = static_cast<long long>(blockIdx.y) * a.slab;
  const long long r1 = r0 + a.slab < a.m ? r0 + a.slab : a.m;
  const int count = a.n - col < 8 ? (a.n - col < 0 ? 0 : a.n - col) : 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto unpack8 = [](uint4 t, float* f) {
    const float2 f0 = unpack_bf16(t.x), f1 = unpack_bf16(t.y), f2 = unpack_bf16(t.z), f3 = unpack_bf16(t.w);
    f[0] = f0.x; f[1] = f0.y; f[2] = f1.x; f[3] = f1.y;
    f[4] = f2.x; f[5] = f2.y; f[6] = f3.x; f[7] = f3.y;
  };
  auto finish = [&](long long r, float* d, const float* z) {  // one row's 8 columns
    if (ACT != kActNone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] *= lin_act_grad<ACT>(z[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] *= a.alpha;
      s[i] += d[i];
    }
    if (a.dz) {  // columns of the padding get zeros, up to `low` with remainders (a product's steps run through them)
      const uint4 hi =
          make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
      *reinterpret_cast<uint4*>(a.dz + r * a.dz_ld + col) = hi;
      if (a.low) {  // what the rounding left, rounded in turn
        float h[8];
        unpack8(hi, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fabsf(h[i]) <= 3.4e38f ? d[i] - h[i] : 0.f;  // none for infinities and NaN
        *reinterpret_cast<uint4*>(a.dz + r * a.dz_ld + a.low + col) =
            make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
      }
    }
  };
  if (count == 8 && a.dout_vec && (ACT == kActNone || a.z_vec)) {
    // Four rows' loads in flight per warp and the registers that takes (two blocks per SM): 4608 x 9216 with GELU in
    // about 57 us (255 MB, floor 39). Three blocks per SM spill: 94; two rows and four blocks 60; one row and six 84.
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(a.dout) + col;
    const __nv_bfloat16* zp = a.z + col;
    for (long long r = r0 + warp; r < r1; r += 32) {
      uint4 dv[4], zv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = r + 8 * u < r1;
        dv[u] = in ? __ldcs(reinterpret_cast<const uint4*>(dout + (r + 8 * u) * a.dout_ld)) : make_uint4(0, 0, 0, 0);
        zv[u] = in && ACT != kActNone ? __ldcs(reinterpret_cast<const uint4*>(zp + (r + 8 * u) * a.z_ld))
                                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r + 8 * u >= r1) break;
        float d[8], z[8];
        unpack8(dv[u], d);
        unpack8(zv[u], z);
        finish(r + 8 * u, d, z);
      }
    }
  } else if (count > 0 || col < a.low) {
    for (long long r = r0 + warp; r < r1; r += 8) {
      float d[8], z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = i < count ? lin_load(a.dout, r * a.dout_ld + col + i, a.dout_f32) : 0.f;
        z[i] = i < count && ACT != kActNone ? __bfloat162float(a.z[r * a.z_ld + col + i]) : 0.f;
      }
      finish(r, d, z);
    }
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

// How one product's tiles are dealt out, from its sizes alone (k_blocks
// counts k twice where A has low halves). Costs in clocks at 1.9 GHz: a 64-deep
// step of a 256 x 256 tile takes about 750 with all pairs at work, a part
// 1500 more for filling and emptying its pipeline, the second launch 5000, and
// the parts' sums go to L2 and back at about 4000 bytes per clock.
LinPlan plan_linear(long long m, long long n, long long k_blocks) {
  LinPlan p{};
  p.m_tiles = static_cast<int>((m + 255) / 256);
  p.n_tiles = static_cast<int>((n + 255) / 256);
  const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
  p.part_rb = static_cast<int>(m < 256 ? (m + 31) / 32 : 8);
  p.part_cb = static_cast<int>(n < 256 ? (n + 31) / 32 : 8);
  p.whole = static_cast<int>(tiles);
  p.waves = static_cast<int>((tiles + kLinPairs - 1) / kLinPairs);
  const int rest = static_cast<int>(tiles % kLinPairs);
  if (rest == 0) return p;
  double best = 750.0 * k_blocks + 1500;
  // at least 4 steps to a part, and at most two rounds of parts (more parts
  // only add traffic)
  for (long long parts = 2; parts * 4 <= k_blocks && rest * parts <= 2 * kLinPairs; ++parts) {
    const long long rounds = (rest * parts + kLinPairs - 1) / kLinPairs;
    const double bytes = 2.0 * rest * parts * p.part_rb * p.part_cb * kLinBox;
    const double cost = rounds * (750.0 * ((k_blocks + parts - 1) / parts) + 1500) + 5000 + bytes / 4000;
    if (cost < best) {
      best = cost;
      p.cut = rest;
      p.parts = static_cast<int>(parts);
    }
  }
  if (p.cut) {
    p.whole = static_cast<int>(tiles) - rest;
    p.waves = p.whole / kLinPairs;
    p.partial_bytes = static_cast<size_t>(p.cut) * p.parts * p.part_rb * p.part_cb * kLinBox;
  }
  return p;
}

template <bool AMN, bool BMN, bool FINE, bool FULL>
static int launch_lin_one(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo, const CUtensorMap& mr,
                          const LinGemmArgs& g, cudaStream_t s) {
  static int pairs_dev[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return -1;
  int& pairs = pairs_dev[dev];
  auto kernel = linear_gemm_kernel<AMN, BMN, FINE, FULL>;
  if (pairs == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem) != cudaSuccess) return -1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * kLinPairs);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kLinSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return -1;
    pairs = n < kLinPairs ? n : kLinPairs;
  }
  const int grid = g.pairs < pairs ? g.pairs : pairs;
  const cudaError_t e = launch_kernel(kernel, dim3(2 * grid), dim3(kLinThreads), kLinSmem, s, 2, ma, mb, mo, mr, g);
  note_launch();
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

// Whether TMA can take a matrix's rows: 16-byte aligned address and pitch, and
// a width of whole 16-byte pieces (a store clips a row to those: past an odd
// width it would write zeros).
static bool tma_rows_ok(const void* p, long long ld, long long n, int f32) {
  const int size = f32 ? 4 : 2;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0 && (n * size) % 16 == 0;
}

int launch_linear_gemm(const LinOperand& a, const LinOperand& b, int k, const LinEpi& epi, float* partial,
                       cudaStream_t s) {
  const int kb = (k + 63) / 64;
  const int passes = a.low ? 2 : 1;
  const LinPlan plan = plan_linear(epi.m, epi.n, static_cast<long long>(kb) * passes);
  CUtensorMap ma, mb;
  // box: 64 k x 128 rows of a k-contiguous operand, 64 rows x 64 k of a
  // row-contiguous one; A's low halves follow its high ones a.low columns on
  const uint64_t a_inner = static_cast<uint64_t>(a.mn_major ? epi.m : k) + a.low;
  if (make_map_2d(&ma, a.data, a_inner, a.mn_major ? k : epi.m, static_cast<uint64_t>(a.ld) * 2, 64,
                  a.mn_major ? 64 : 128) ||
      make_map_2d(&mb, b.data, b.mn_major ? epi.n : k, b.mn_major ? k : epi.n, static_cast<uint64_t>(b.ld) * 2, 64,
                  b.mn_major ? 64 : 128))
    return -2;
  LinGemmArgs g{};
  g.m_tiles = plan.m_tiles;
  g.n_tiles = plan.n_tiles;
  g.k_blocks = kb;
  g.a_low = a.low;
  g.waves = plan.waves;
  g.whole = plan.whole;
  g.cut = plan.cut;
  g.parts = plan.parts;
  g.n_fastest = epi.n <= epi.m;  // the smaller operand stays in L2, the larger streams through once
  const int most = plan.waves > 0 ? plan.whole : plan.cut * plan.parts;
  g.pairs = most < kLinPairs ? most : kLinPairs;
  g.partial = partial;
  g.part_rb = plan.part_rb;
  g.part_cb = plan.part_cb;
  g.epi = epi;
  CUtensorMap mo = ma, mr = ma;  // not read unless epi.tma
  g.epi.tma = tma_rows_ok(epi.out, epi.out_ld, epi.n, epi.out_f32) &&
              (!epi.res || tma_rows_ok(epi.res, epi.res_ld, epi.n, epi.res_f32)) &&
              (!epi.z || tma_rows_ok(epi.z, epi.z_ld, epi.n, 0));
  if (g.epi.tma && (make_map_rows32(&mo, epi.out, epi.n, epi.m, epi.out_ld, epi.out_f32) ||
                    (epi.res && make_map_rows32(&mr, epi.res, epi.n, epi.m, epi.res_ld, epi.res_f32))))
    return -2;
  int rc;
  const bool fine = epi.out_f32, full = epi.bias || epi.z || epi.act != kActNone;
  if (a.low && (!fine || full)) return -2;  // low halves are summed in registers, without an epilogue
  if (a.mn_major) {
    if (full) return -2;
    rc = fine ? launch_lin_one<true, true, true, false>(ma, mb, mo, mr, g, s)
              : launch_lin_one<true, true, false, false>(ma, mb, mo, mr, g, s);
  } else if (b.mn_major) {
    if (full) return -2;
    rc = fine ? launch_lin_one<false, true, true, false>(ma, mb, mo, mr, g, s)
              : launch_lin_one<false, true, false, false>(ma, mb, mo, mr, g, s);
  } else if (full) {
    rc = fine ? launch_lin_one<false, false, true, true>(ma, mb, mo, mr, g, s)
              : launch_lin_one<false, false, false, true>(ma, mb, mo, mr, g, s);
  } else {
    rc = fine ? launch_lin_one<false, false, true, false>(ma, mb, mo, mr, g, s)
              : launch_lin_one<false, false, false, false>(ma, mb, mo, mr, g, s);
  }
  if (rc || !plan.cut) return rc;
  const cudaError_t e =
      launch_kernel(linear_finish_kernel, dim3(plan.part_rb * plan.part_cb, plan.cut), dim3(256), 0, s, 1, g);
  note_launch();
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

template <int NB>
static cudaError_t launch_rows_nb(const __nv_bfloat16* x, long long x_ld, const __nv_bfloat16* w, long long w_ld, int k,
                                  const LinEpi& e, cudaStream_t s) {
  const dim3 grid((e.n + 15) / 16, (e.m + 8 * NB - 1) / (8 * NB));
  if (grid.x * grid.y < 4 * kLinSms && k >= 2048)
    return launch_kernel(linear_rows_kernel<NB, 16>, grid, dim3(512), 0, s, 1, x, x_ld, w, w_ld, k, e);
  return launch_kernel(linear_rows_kernel<NB, 8>, grid, dim3(256), 0, s, 1, x, x_ld, w, w_ld, k, e);
}

// 16 rows or fewer, or a small problem: blocks of 32 rows x 16 columns for about one round over the SMs, and not
// much re-reading of the weights. Measured on one B200 (us, back to back, against linear_gemm_kernel): 8 x 27648 x 3072
// 29 (floor 26) against 50; 16 rows of it 33 against 38, 32 rows 54 against 39; 96 x 640 x 640 3.3 against 7.5;
// 96 x 3072 x 1024 7.5 against 11, 96 x 3072 x 3072 19 against 13; 256 x 1024 x 256 5.1 against 6.3, 512 rows of it
// 9.2 against 6.3; 4608 x 16 x 3072 5.6 against 13. At the border, four sets of operands in turn: volume 9.0M (96 x 3072 x 1024) 7.5
// against 10.9, 10.0M (256 x 1024 x 1280) 9.4 against 10.0, 12.0M (64 x 3072 x 2048) 12.0 against 11.3, 13.5M
// (4608 x 32 x 3072) 14.8 against 13.2, 16.0M (256 x 1024 x 2048) 14.2 against 10.5; columns fill the blocks of 16 worse
// at 4608 x 24 x 3072 (10.1M), 14.5 against 13.2.
bool linear_rows_fit(int m, int n, int k) {
  if (m <= 16) return true;
  const long long row_blocks = (m + 31) / 32;
  return row_blocks * ((n + 15) / 16) <= 640 && row_blocks * n * k <= 12ll << 20;
}

int launch_linear_rows(const __nv_bfloat16* x, long long x_ld, const __nv_bfloat16* w, long long w_ld, int k,
                       const LinEpi& e, cudaStream_t s) {
  const cudaError_t rc = e.m <= 8    ? launch_rows_nb<1>(x, x_ld, w, w_ld, k, e, s)
                         : e.m <= 16 ? launch_rows_nb<2>(x, x_ld, w, w_ld, k, e, s)
                                     : launch_rows_nb<4>(x, x_ld, w, w_ld, k, e, s);
  note_launch();
  return (rc == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

// Rows per block of linear_dz_kernel: about four blocks per SM, slabs a
// multiple of the 32 rows that a block's warps take at a time.
int lin_dz_slab(long long m, int n) {
  const long long col_blocks = (n + 255) / 256;
  long long slabs = (4 * kLinSms + col_blocks - 1) / col_blocks;
  const long long most = (m + 31) / 32;
  if (slabs > most) slabs = most;
  if (slabs < 1) slabs = 1;
  const long long slab = (m + slabs - 1) / slabs;
  return static_cast<int>((slab + 31) / 32 * 32);
}

int launch_linear_dz(const LinDzArgs& a, float* dbias, cudaStream_t s) {
  const int slabs = static_cast<int>((a.m + a.slab - 1) / a.slab);
  auto kernel = a.act == kActNone   ? linear_dz_kernel<kActNone>
                : a.act == kActSilu ? linear_dz_kernel<kActSilu>
                                    : linear_dz_kernel<kActGelu>;
  cudaError_t e = launch_kernel(kernel, dim3((a.n + 255) / 256, slabs), dim3(256), 0, s, 1, a);
  note_launch();
  if (e == cudaSuccess && dbias) {
    e = launch_kernel(linear_dbias_kernel, dim3((a.n + 255) / 256), dim3(256), 0, s, 1,
                      static_cast<const float*>(a.col_part), slabs, a.n, dbias);
    note_launch();
  }
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

}  // namespace klein
