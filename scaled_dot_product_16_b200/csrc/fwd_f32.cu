// fwd_f32.cu -- attention forward in float32 on the CUDA cores (the ATTN_F32 path).
//
// O = softmax(scale * Q K^T + mask) V with per-row max / sum statistics, for dense BHSD or
// packed TND batches, GQA/MQA and causal masks ("aclnnFlashAttentionVarLenScore", 功能说明
// and 约束说明; formula of "paddle.nn.functional.sparse_attention"). The torch.nn.attention
// blog notes that fp32 inputs leave the fast flash path; here fp32 keeps full fp32 FMA
// arithmetic (no TF32), so the result stays within 1e-5 of the exact value.
//
// Tiling: a block owns 32 query rows of one (sequence, head); its 8 warps own 4 rows each.
// Key/value tiles of 32 rows are staged in shared memory; lane = key for the scores and
// lane = head-dim column for the P.V accumulation. The softmax is the online (streaming)
// form: the running maximum and sum are rescaled when the maximum grows. attn_fwd_sinks leaves out
// the key tiles between the first keys and the block's window.
//
// The tiles come by asynchronous copies, the next one while the current one is multiplied: with plain
// loads a block of few key tiles spent most of its time waiting for them (2 x 4 x 333 x 80, window 128:
// 121 us, now 23). Where rows are whole 16-byte chunks a row is one bulk copy, issued by four lanes of
// each warp: per-thread copies took every warp 2,000 of a tile's 7,000 cycles to issue (28 us; all rows
// from one warp: 33), the queries with the first tile (25 -> 22 us). Rows are padded to whole 16-byte chunks, so that
// queries and keys are read four columns at a time, and the weights four rows at a time: the loop is
// bound by shared-memory reads otherwise. The order of every sum is that of one column, and one key,
// after the other.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace sdpa {
namespace {

constexpr int kBM = 32;       // query rows per block
constexpr int kBN = 32;       // keys per tile
// Warps of a block, 4 rows each. 4 warps of 8 rows read K less often but hide less (1.2 to 1.5 times the
// time), 16 of 2 rows are bound by the reads of K (1.3 to 1.6 times).
constexpr int kWarps = 8;
constexpr int kRowsPerWarp = kBM / kWarps;

using namespace sm100;

constexpr uint64_t kWaitNs = 1000ull * 1000ull * 1000ull;  // bound on the wait for a tile

// 4 bytes to shared memory, or a zero where !ok (src is then not read)
__device__ __forceinline__ void stage(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 4 : 0) : "memory");
}

// kBN rows of D columns into rows of `ld` floats whose columns up to a multiple of 4 become zeros; rows
// from `rows` on become zeros. A warp copies kBN / kWarps rows in a row, all at once where they have no more columns
// than it has lanes (2 x 8 x 1,128, head size 1: 266 us with a row at a time and the kernel of head sizes up to 64, 168 so).
__device__ __forceinline__ void stage_tile(float* dst, int ld, const float* src, int64_t stride, int rows, int D) {
  constexpr int kRows = kBN / kWarps;
  const int r0 = (threadIdx.x >> 5) * kRows, lane = threadIdx.x & 31;
  auto one = [&](int r, int c) {
    const bool ok = r < rows && c < D;
    stage(dst + r * ld + c, ok ? src + r * stride + c : src, ok);
  };
  if (D <= 8) {
    const int l = D <= 4 ? 2 : 3, r = lane >> l;
    if (r < kRows) one(r0 + r, lane & ((1 << l) - 1));
  } else {
    const int D4 = (D + 3) / 4 * 4;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      for (int c = lane; c < D4; c += 32) one(r0 + r, c);
  }
}
static_assert(kBN / kWarps * 8 <= 32, "rows of up to 8 columns at once");

__device__ __forceinline__ bool wait_tile(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, parity, 20000))
    if (globaltimer_ns() - t0 > kWaitNs) return false;
  return true;
}

// Three blocks an SM at head sizes up to 64, whose tiles leave the shared memory for it (4 x 16 x 1,024, window
// 512: 487 -> 453 us; with four registers spill: 502).
// VEC: rows of q, k and v are whole 16-byte chunks. The others have a kernel of their own, as both kinds of copies in
// one take registers that the loop needs (2 x 8 x 1,128, head size 4: 200 us, apart 180).
template <int DMAX, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, DMAX <= 64 ? 3 : 2) fwd_f32_kernel(FwdArgs a, int tiles_per_seq, int x0) {
  extern __shared__ __align__(16) float smem[];
  const int D = a.D, Dv = a.Dv;
  const int D4 = (D + 3) / 4 * 4, Dv4 = (Dv + 3) / 4 * 4;
  const int ldk = (D4 / 4 | 1) * 4;  // row of the K tile, an odd number of chunks: lane-strided 16-byte reads avoid bank conflicts
  float* sQ = smem;                       // [kBM][D4]
  float* sP = sQ + kBM * D4;              // [kWarps][kBN][kRowsPerWarp]
  float* sK = sP + kWarps * kRowsPerWarp * kBN;  // [2][kBN][ldk]
  float* sV = sK + 2 * kBN * ldk;         // [2][kBN][Dv4]
  __shared__ int s_info[4];
  __shared__ __align__(8) uint64_t s_full[2];  // the tile of each buffer has come (16-byte rows)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Blocks start in the order of their index: the heads of a query tile side by side, and the last tiles of
  // the sequences first, as a causal mask gives those the most keys and a long block that starts late ends
  // late (2 x 8 x 1,128 x 128, causal: 390 -> 266 us).
  const int xb = blockIdx.x / a.Nq, h = blockIdx.x - xb * a.Nq;
  const int x = x0 + xb;
  const int g = h / (a.Nq / a.Nkv);

  // ---- which (sequence, query tile) this block owns -------------------------------------
  if (warp == 0) {
    int b, t, ok;
    if (a.layout == ATTN_BHSD) {
      t = x / a.B;
      b = x - t * a.B;
      t = tiles_per_seq - 1 - t;
      ok = 1;
    } else {
      bool bad;
      ok = warp_find_tile(a.cu_q, a.B, a.Sq, kBM, x, &b, &t, a.status, &bad);
      if (ok) {
        int qs, ql;
        seq_span(a.cu_q, b, &qs, &ql);
        t = (ql + kBM - 1) / kBM - 1 - t;
      }
      if (!ok && !bad && h == 0) {
        // a block past the last tile checks the key-side lengths for everyone
        int seq, tis;
        bool bad2;
        warp_find_tile(a.cu_kv, a.B, a.Skv, 1 << 30, 1 << 30, &seq, &tis, a.status, &bad2);
      }
    }
    if (lane == 0) {
      mbar_init(smem_u32(&s_full[0]), 1);
      mbar_init(smem_u32(&s_full[1]), 1);
      fence_mbar_init();
      s_info[0] = ok;
      s_info[1] = b;
      s_info[2] = t;
    }
  }
  __syncthreads();
  if (!s_info[0]) return;
  const int b = s_info[1], qt = s_info[2];

  int q0, sq, k0, sk;  // token offsets and lengths of this sequence
  if (a.layout == ATTN_BHSD) {
    q0 = 0;
    sq = a.Sq;
    k0 = 0;
    sk = a.Skv;
  } else {
    seq_span(a.cu_q, b, &q0, &sq);
    seq_span(a.cu_kv, b, &k0, &sk);
    if (k0 < 0 || sk < 0 || k0 + sk > a.Skv) {
      if (threadIdx.x == 0) report(a.status, ATTN_ERR_DATA);
      return;
    }
  }
  const float* Q = (const float*)a.q;
  const float* K = (const float*)a.k;
  const float* V = (const float*)a.v;
  // element (token i of this sequence, head, d)
  auto qoff = [&](int i) -> int64_t {
    return a.layout == ATTN_BHSD ? (((int64_t)b * a.Nq + h) * a.Sq + i) * D
                                 : ((int64_t)(q0 + i) * a.Nq + h) * D;
  };
  auto kvoff = [&](int j) -> int64_t {
    return a.layout == ATTN_BHSD ? (((int64_t)b * a.Nkv + g) * a.Skv + j) * D
                                 : ((int64_t)(k0 + j) * a.Nkv + g) * D;
  };
  // value rows and output rows have Dv columns
  auto voff = [&](int j) -> int64_t {
    return a.layout == ATTN_BHSD ? (((int64_t)b * a.Nkv + g) * a.Skv + j) * Dv
                                 : ((int64_t)(k0 + j) * a.Nkv + g) * Dv;
  };
  auto ooff = [&](int i) -> int64_t {
    return a.layout == ATTN_BHSD ? (((int64_t)b * a.Nq + h) * a.Sq + i) * Dv
                                 : ((int64_t)(q0 + i) * a.Nq + h) * Dv;
  };
  const uint8_t* mrow0 = a.mask != nullptr ? a.mask + (int64_t)b * a.mask_bs : nullptr;

  const int row0 = qt * kBM;
  const int nrows = min(kBM, sq - row0);
  constexpr int kLaneRows = kBN / kWarps;  // VEC: the first lanes of each warp copy a row each
  static_assert(kBN == kBM, "rows of a tile");
  const int64_t k_stride = a.layout == ATTN_BHSD ? D : (int64_t)a.Nkv * D;
  const int64_t v_stride = a.layout == ATTN_BHSD ? Dv : (int64_t)a.Nkv * Dv;
  auto fetch = [&](int j0, int buf, int bytes) {  // the key tile at j0; `bytes` more come to its barrier
    float* kt = sK + buf * kBN * ldk;
    float* vt = sV + buf * kBN * Dv4;
    if constexpr (!VEC) {
      stage_tile(kt, ldk, K + kvoff(j0), k_stride, sk - j0, D);
      stage_tile(vt, Dv4, V + voff(j0), v_stride, sk - j0, Dv);
    } else {
      // Value rows behind the last key become zeros: their weights are 0, but what lies there may be
      // anything. (Keys there are not looked at.)
      const int rows = min(kBN, sk - j0), r = warp * kLaneRows + lane;
      const uint32_t bar = smem_u32(&s_full[buf]);
      if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, rows * (D + Dv) * 4 + bytes);
      if (lane < kLaneRows) {
        if (r < rows) {
          bulk_load(smem_u32(kt + r * ldk), K + kvoff(j0) + r * k_stride, D * 4, bar);
          bulk_load(smem_u32(vt + r * Dv4), V + voff(j0) + r * v_stride, Dv * 4, bar);
        } else {
          for (int c = 0; c < Dv; c += 4) *reinterpret_cast<float4*>(vt + r * Dv4 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      __syncwarp();
    }
  };

  // keys needed by the tile: from the first row's first visible key to the last row's last
  const int kv_end = visible_end(a.mask_mode, row0 + nrows - 1, sq, sk, a.next);
  const bool sinks = a.mask_mode == kMaskSinks;
  const int kv_begin = (sinks ? window_begin(row0, sq, sk, a.pre) : visible_begin(a.mask_mode, row0, a.pre)) / kBN * kBN;
  // attn_fwd_sinks: the tiles of the first keys come before those of the window
  const int sink_end = sinks ? (min(a.sinks, kv_begin) + kBN - 1) / kBN * kBN : 0;

  constexpr int DT = DMAX / 32;  // head-dim columns per lane
  float acc[kRowsPerWarp][DT];
  float m[kRowsPerWarp], l[kRowsPerWarp];
  int vbeg[kRowsPerWarp], vend[kRowsPerWarp];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    const int i = row0 + warp * kRowsPerWarp + r;
    vend[r] = i < sq ? visible_end(a.mask_mode, i, sq, sk, a.next) : 0;
    vbeg[r] = sinks ? window_begin(i, sq, sk, a.pre) : visible_begin(a.mask_mode, i, a.pre);
#pragma unroll
    for (int t = 0; t < DT; ++t) acc[r][t] = 0.f;
  }

  auto after = [&](int j0) { return j0 + kBN == sink_end ? kv_begin : j0 + kBN; };
  int buf = 0, it = 0;
  const int j_first = sink_end > 0 ? 0 : kv_begin;
  if (j_first < kv_end) {
    if (VEC && lane < kLaneRows) {  // Q with the first tile
      const int r = warp * kLaneRows + lane;
      if (r < nrows)
        bulk_load(smem_u32(sQ + r * D4), Q + qoff(row0 + r), D * 4, smem_u32(&s_full[0]));
      else
        for (int c = 0; c < D; c += 4) *reinterpret_cast<float4*>(sQ + r * D4 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncwarp();
    // rows past the sequence's end become zeros
    if constexpr (!VEC) stage_tile(sQ, D4, Q + qoff(row0), a.layout == ATTN_BHSD ? D : (int64_t)a.Nq * D, nrows, D);
    fetch(j_first, 0, nrows * D * 4);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int j0 = j_first; j0 < kv_end; j0 = after(j0), buf ^= 1, ++it) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    const bool come = !VEC || wait_tile(smem_u32(&s_full[buf]), (it >> 1) & 1);
    // this tile is there (and Q, on the first pass), and the last one is consumed
    if (__syncthreads_or(!come)) {
      if (threadIdx.x == 0) report(a.status, ATTN_ERR_TIMEOUT);
      wait_tile(smem_u32(&s_full[buf]), (it >> 1) & 1);  // no copy outlives the block
      return;
    }
    if (after(j0) < kv_end) fetch(after(j0), buf ^ 1, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");

    // scores: lane = key j0 + lane, one value per row of this warp
    float s[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) s[r] = 0.f;
    const float* kr = sK + buf * kBN * ldk + lane * ldk;
    const float* qr = sQ + warp * kRowsPerWarp * D4;
#pragma unroll 8
    for (int d = 0; d < D4; d += 4) {
      const float4 kv = *reinterpret_cast<const float4*>(kr + d);
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const float4 qv = *reinterpret_cast<const float4*>(qr + r * D4 + d);
        s[r] = fmaf(qv.x, kv.x, s[r]);
        s[r] = fmaf(qv.y, kv.y, s[r]);
        s[r] = fmaf(qv.z, kv.z, s[r]);
        s[r] = fmaf(qv.w, kv.w, s[r]);
      }
    }
    const int j = j0 + lane;
    float* pw = sP + warp * kRowsPerWarp * kBN;
    // the rows' reductions side by side, without branches between them
    float pr[kRowsPerWarp], mx[kRowsPerWarp], ps[kRowsPerWarp], corr[kRowsPerWarp];
    bool vis[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      vis[r] = (j >= vbeg[r] || (sinks && j < a.sinks)) && j < vend[r];
      if (mrow0 != nullptr && vis[r]) vis[r] = mrow0[(int64_t)(row0 + warp * kRowsPerWarp + r) * a.mask_rs + j] == 0;
      s[r] = vis[r] ? s[r] * a.scale : -INFINITY;
      mx[r] = s[r];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], o));
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const float mnew = fmaxf(m[r], mx[r]);
      const float muse = mnew == -INFINITY ? 0.f : mnew;
      const float e = expf(s[r] - muse), c = expf(m[r] - muse);  // of -inf: 0
      pr[r] = ps[r] = vis[r] ? e : 0.f;
      corr[r] = c;
      m[r] = mnew;
#pragma unroll
      for (int t = 0; t < DT; ++t) acc[r][t] *= c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) ps[r] += __shfl_xor_sync(0xffffffffu, ps[r], o);
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) l[r] = fmaf(l[r], corr[r], ps[r]);
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; r += 4)
      *reinterpret_cast<float4*>(pw + lane * kRowsPerWarp + r) = make_float4(pr[r], pr[r + 1], pr[r + 2], pr[r + 3]);
    __syncwarp();
    // P.V: lane owns head-dim columns lane, lane+32, ...
    const float* vt = sV + buf * kBN * Dv4;
#pragma unroll 8
    for (int jj = 0; jj < kBN; ++jj) {
      const float* vr = vt + jj * Dv4;
      float vv[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) vv[t] = (lane + 32 * t) < Dv ? vr[lane + 32 * t] : 0.f;
      float p[kRowsPerWarp];
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; r += 4)
        *reinterpret_cast<float4*>(p + r) = *reinterpret_cast<const float4*>(pw + jj * kRowsPerWarp + r);
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[r][t] = fmaf(p[r], vv[t], acc[r][t]);
    }
  }

  // ---- epilogue ---------------------------------------------------------------------------
  float* O = (float*)a.out;
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const int i = row0 + warp * kRowsPerWarp + r;
    if (i >= sq) continue;  // warp-uniform
    const bool any = l[r] > 0.f;
    const float m_loc = any ? m[r] : -INFINITY;
    const float l_loc = l[r];
    float f_o = any ? 1.f / l[r] : 0.f;
    float f_prev = 0.f;
    int64_t o;
    if (a.acc_mode == 0) {
      o = ooff(i);
      if (lane == 0 && a.smax != nullptr) {
        const int64_t so = a.layout == ATTN_BHSD ? ((int64_t)b * a.Nq + h) * a.Sq + i
                                                 : (int64_t)(q0 + i) * a.Nq + h;
        a.smax[so] = m_loc;
        a.ssum[so] = l_loc;
      }
    } else {
      // accumulator in the merge layouts: BHSD -> output [Sq, B, Nq*D] (SBH), statistics
      // [B, Nq, Sq, 8]; TND -> output [T, Nq*D], statistics [T, Nq, 8]. Lanes 0-7 update the
      // 8 statistic lanes ("npu_ring_attention_update", 小算子等价计算逻辑); lane 0's factors
      // rescale the output row.
      o = a.layout == ATTN_BHSD ? (((int64_t)i * a.B + b) * a.Nq + h) * D : qoff(i);
      const int64_t so = (a.layout == ATTN_BHSD ? ((int64_t)b * a.Nq + h) * a.Sq + i
                                                : (int64_t)(q0 + i) * a.Nq + h) * 8;
      float ps2 = 0.f, cs2 = 0.f, nl = 0.f;
      if (lane < 8) {
        if (a.acc_mode == 1) {
          a.smax[so + lane] = m_loc;
          a.ssum[so + lane] = l_loc;
          cs2 = l_loc;
          nl = l_loc;
        } else {
          const float pm = a.smax[so + lane], ps = a.ssum[so + lane];
          const float mk = fmaxf(pm, m_loc);
          if (mk != -INFINITY) {
            ps2 = ps * expf(pm - mk);
            cs2 = l_loc * expf(m_loc - mk);
          }
          nl = ps2 + cs2;
          a.smax[so + lane] = mk;
          a.ssum[so + lane] = nl;
        }
      }
      ps2 = __shfl_sync(0xffffffffu, ps2, 0);
      cs2 = __shfl_sync(0xffffffffu, cs2, 0);
      nl = __shfl_sync(0xffffffffu, nl, 0);
      const float inv = nl != 0.f ? 1.f / nl : 0.f;
      f_prev = a.acc_mode == 1 ? 0.f : ps2 * inv;
      f_o = a.acc_mode == 1 ? f_o : f_o * cs2 * inv;
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const int d = lane + 32 * t;
      if (d < Dv) {
        float v = acc[r][t] * f_o;
        if (a.acc_mode == 2) v = fmaf(O[o + d], f_prev, v);
        O[o + d] = v;
      }
    }
  }
}

// Shared memory of a block, for head sizes rounded up to multiples of 4.
constexpr int smem_bytes(int D4, int Dv4) {
  return (int)sizeof(float) * (kBM * D4 + kBM * kBN + 2 * kBN * ((D4 / 4 | 1) * 4) + 2 * kBN * Dv4);
}

template <int DMAX, bool VEC>
cudaError_t launch_kernel(const FwdArgs& a, cudaStream_t st) {
  const int smem = smem_bytes((a.D + 3) / 4 * 4, (a.Dv + 3) / 4 * 4);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fwd_f32_kernel<DMAX, VEC>), smem_bytes(DMAX, DMAX), ready);
  if (e != cudaSuccess) return e;
  int tiles_per_seq = 0;
  int64_t gx;
  if (a.layout == ATTN_BHSD) {
    tiles_per_seq = (a.Sq + kBM - 1) / kBM;
    gx = (int64_t)a.B * tiles_per_seq;
  } else {
    gx = (a.Sq + kBM - 1) / kBM + a.B;  // upper bound on the tiles of a packed batch
  }
  if (gx <= 0) return cudaSuccess;
  if (gx > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // as many query tiles a launch as a grid holds with all their heads (one launch but for 2^31 blocks and more)
  const int64_t per = 0x7fffffff / a.Nq;
  for (int64_t x0 = 0; x0 < gx; x0 += per) {
    const unsigned grid = (unsigned)((gx - x0 < per ? gx - x0 : per) * a.Nq);
    fwd_f32_kernel<DMAX, VEC><<<grid, kWarps * 32, smem, st>>>(a, tiles_per_seq, (int)x0);
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess) return launched;
  }
  return cudaSuccess;
}

template <int DMAX>
cudaError_t launch_dmax(const FwdArgs& a, cudaStream_t st) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  const bool vec = (all & 15u) == 0 && a.D % 4 == 0 && a.Dv % 4 == 0;
  return vec ? launch_kernel<DMAX, true>(a, st) : launch_kernel<DMAX, false>(a, st);
}

}  // namespace

cudaError_t launch_fwd_f32(const FwdArgs& a, cudaStream_t st) {
  if (a.D <= 32) return launch_dmax<32>(a, st);
  if (a.D <= 64) return launch_dmax<64>(a, st);
  if (a.D <= 96) return launch_dmax<96>(a, st);
  if (a.D <= 128) return launch_dmax<128>(a, st);
  return launch_dmax<256>(a, st);
}

}  // namespace sdpa
