// block.cuh -- the norms before and after a block, fused with its gate and its
// scales, and the norms that keep their input as an 8-bit checkpoint.
//
//   z = x rstd1 W1'          rstd1 = 1/sqrt(mean x^2 + eps), W1' = w1 + offset
//   h = a r + b g z          gate g: one row, one row per R rows, or one per row
//   y = h rstd2 W2'          rstd2 = 1/sqrt(mean h^2 + eps)
//
// With neither a first norm nor a gate this is the fused add + RMSNorm, and
// without a residual the RMSNorm; with LN the norm of h = x is LayerNorm.  Those
// forms serve the checkpointed calls of the three norms.
//
// Both directions are bound by memory: about 12 and 30 floating-point
// operations an element against 4 and 6 streamed values.  Every row is read
// once and written once; what is left is to keep the copies running.  So, as
// in the other row kernels: persistent row groups, rows brought in by bulk
// copies through a ring of shared-memory stages, 16 to 32 columns a thread whose
// per-column values (W2', C = b g W1' and the gradients' sums) stay in
// registers for the whole launch, FP32 arithmetic on pairs.
//
// The forward takes two sums that depend on one another (rstd1, then the sum
// of h^2), one barrier each; h stays in registers from the second pass to the
// third.  Expanding sum h^2 into sums over x and r would save a barrier but
// lose precision quadratically where a r and b g z cancel.
//
// The backward takes one pass and one barrier: with g2 = dy W2', C x streamed,
//   dh = rstd2 g2 + dh_out - k h,     k = rstd2^3 sum(g2 h) / N
//   sum dh C x = sum (rstd2 g2 + dh_out) C x - k sum h C x
// so the second norm's row constant is known from three sums of one pass (it is
// linear in dh, so the error stays that of dh itself: relative to the terms).
//   d residual = a dh;  dx = rstd1 (dh C - x rstd1^2 sum(dh C x) / N)
//   dw2 = sum dy h rstd2;  A = sum dh x rstd1 gives dw1 = b g A and dg = b W1' A.
//
// A thread owns 16 to 32 columns of its CTA's slice (fwd_cta, bwd_cta), a warp 32
// times as many, consecutive.
// Each kernel comes in an aligned form (ALN: rows start on 16 bytes, N a
// multiple of 16 bytes of elements; a thread owns 16-byte chunks 32 lanes apart)
// and a general one (any N, stride, alignment; a thread owns single columns 32
// apart).  In the general form a row's copy is rounded out to 16 bytes, except
// where that would leave the matrix (near its first and last row): there it is
// rounded in, and the few elements at the edge are read from global memory.
// CL: a row is split over a thread-block cluster, whose CTAs exchange their sums
// through distributed shared memory.
//
// FORM fixes which norms there are, so that the row loop holds no test of it;
// kDynamic (general form) decides at run time.
#pragma once

#include <initializer_list>

#include "../kernels.cuh"
#include "block.h"
#include "ckpt.cuh"

namespace gb300norm {

constexpr int kSliceCols = 8192;    // columns a CTA takes at most
constexpr int kBlockMaxStages = 16;
constexpr int kBlockHeader = 128;   // mbarriers

// kNorm: the norm of h alone, without x, gate and scales (RMSNorm and fused add).
enum BlockForm : int { kBoth = 0, kPre = 1, kPost = 2, kLn = 3, kDynamic = 4, kNorm = 5 };

// Columns a thread owns, and the threads and CTAs the registers are bounded for:
// 512 x 1 or 256 x 2 give up to 128 registers a thread (16 warps an SM), 640 x 1
// and 32 x 20 up to 96 (20 warps), 256 x 1 up to 255 (8 warps).
//  * backward of h's norm with x (kBoth, kPre): W2', C and both gradients' sums
//    are 128 registers at 32 columns; at 16 columns the rest does not fit in 128.
//    LayerNorm's: 32 columns, its two rows in registers as well (KEEP).
//    The other shape (ALT = 1): 24 columns, where that puts more of the 8 warps to
//    work (5120 columns: 7 in place of 5, 6144: 8 in place of 6; both norms at
//    8192 x 5120 121 -> 101 us).
//  * backward of one norm alone (kNorm, kPost): 16 columns; its two rows kept
//    from the sums to the outputs, or (ALT) read and decoded again with 96
//    registers, where a row's warps then fit an SM more often: 10 warps (5120
//    columns) twice in place of once, RMSNorm 62.9 -> 51.1 us at 8192 x 5120.
//  * forward of one norm alone: 32 columns and two CTAs of 8192 columns an SM, one
//    computing while the other waits at a barrier: RMSNorm with checkpoint at
//    8192 x 8192 73.4 -> 58.0 us, 8192 x 5120 65.2 -> 38.6 us.
//  * the other forwards: 16 columns, or (ALT) 16 in 96 registers: both norms at
//    8192 x 5120 78 -> 57 us, at 8192 x 8192 88 -> 92 us.
//  * the general form: as the forwards above, without checkpoints always in 96
//    registers; 16 columns in every backward: with weight gradients it spills a
//    little at 128 registers and is no slower than 24 or 32 columns at up to 255
//    (4000 x 4100: 108, 108 and 149 us), more warps hiding more.  ALT: 96
//    registers (both norms with checkpoints 4000 x 4100, 9 warps a row: 242 -> 209
//    us a step; 8000 x 1001, 2 warps: 103 -> 115; backward 4096 x 8191, 16 warps:
//    146 -> 184).
//  * rows that one warp holds at 8 columns a thread (kNarrowCta; aligned form): 20
//    CTAs of one warp an SM in place of 8 to 16 hide more of a row's latency,
//    which is most of its time (100000 x 256, both norms: forward 53 -> 40 us,
//    backward frozen 69 -> 53, trained 95 -> 68; 200000 x 128: 101 -> 74, 130 ->
//    97, 181 -> 121).  Not for the weight gradients of kNorm and kLn, whose
//    workspace has 8 partial rows an SM.  With more warps a row it is slower
//    (60000 x 512: backward frozen 59 -> 71).
// A row's columns are dealt to its lanes in the same order whether weight
// gradients are wanted or not: the order of the sums, and so every bit of dx, is
// then the same.
struct BlockCta { int cols, threads, ctas, warps; };   // warps: on an SM
constexpr bool one_norm(int form) { return form == kPost || form == kNorm; }
constexpr BlockCta kNarrowCta{8, 32, 20, 20};   // (ALT = 2)
constexpr BlockCta fwd_cta(int form, bool q8, int alt, bool aln) {
  return alt == 2 ? kNarrowCta
         : one_norm(form) ? BlockCta{32, 256, 2, 16}
         : alt || (!aln && !q8) ? BlockCta{16, 640, 1, 20} : BlockCta{16, 512, 1, 16};
}
constexpr BlockCta bwd_cta(int form, int alt, bool aln) {
  return alt == 2                ? kNarrowCta
         : !aln || one_norm(form) ? (alt ? BlockCta{16, 640, 1, 20} : BlockCta{16, 512, 1, 16})
                                : BlockCta{alt ? 24 : 32, 256, 1, 8};
}

// How the backward meets the gate: none, or one row (kFixed); rows dealt out by
// gate row (kSegments); a gate row for each row (kStreamed).
enum BlockGate : int { kFixed = 0, kStreamed = 1, kSegments = 2 };

// A per-column parameter value of any of the three types.
__device__ __forceinline__ float ld_code(const void* p, int code, int64_t i) {
  if (code == NORM_F32) return static_cast<const float*>(p)[i];
  if (code == NORM_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st_code(void* p, int code, int64_t i, float v) {
  if (code == NORM_F32) static_cast<float*>(p)[i] = v;
  else if (code == NORM_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__host__ __device__ inline int code_size(int code) { return code == NORM_F32 ? 4 : 2; }

// A thread's columns of a row slice and the ways to move them.
template <class T, int NPT, bool ALN>
struct RowIO {
  static constexpr int VEC = 16 / (int)sizeof(T);
  static constexpr int H = VEC / 2;
  static constexpr int WCOLS = 32 * NPT * VEC;   // columns of a warp
  using P = Pack16<T>;
  int c0;     // first chunk (ALN) or first column (general) of this thread
  int nch;    // 16-byte chunks of the slice (ALN)
  int NL;     // columns of the slice
  __device__ __forceinline__ void place(int warp, int lane) { c0 = warp * (ALN ? WCOLS / VEC : WCOLS) + lane; }
  // bytes from a slice's start to this thread's first chunk (column)
  __device__ __forceinline__ int at() const { return c0 * (ALN ? 16 : (int)sizeof(T)); }
  // whether chunk j exists; in the general form a chunk is VEC single columns
  // of which this says whether any does
  __device__ __forceinline__ bool has(int j) const { return ALN ? c0 + j * 32 < nch : c0 + j * VEC * 32 < NL; }
  __device__ __forceinline__ int col(int j, int k) const {
    return ALN ? (c0 + j * 32) * VEC + k : c0 + (j * VEC + k) * 32;
  }
  __device__ __forceinline__ bool valid(int j, int k) const { return ALN ? has(j) : col(j, k) < NL; }
  // general form: every column of chunk j exists, for the whole warp
  __device__ __forceinline__ bool whole(int j) const { return ALN || ((c0 & ~31) + (j + 1) * VEC * 32 <= NL); }

  // `s`: the slice's start in its stage
  __device__ __forceinline__ void load(const unsigned char* s, int j, float2 (&v)[H]) const {
    if constexpr (ALN) {
      P::unpack(reinterpret_cast<const uint4*>(s)[c0 + j * 32], v);
    } else {
      const T* q = reinterpret_cast<const T*>(s) + c0 + j * VEC * 32;
      if (whole(j)) {
#pragma unroll
        for (int h = 0; h < H; ++h) v[h] = make_float2(to_f(q[(2 * h) * 32]), to_f(q[(2 * h + 1) * 32]));
      } else {
#pragma unroll
        for (int h = 0; h < H; ++h)
          v[h] = make_float2(col(j, 2 * h) < NL ? to_f(q[(2 * h) * 32]) : 0.f,
                             col(j, 2 * h + 1) < NL ? to_f(q[(2 * h + 1) * 32]) : 0.f);
      }
    }
  }
  // chunk j of a checkpoint slice: codes, then (at `so`) its scales
  __device__ __forceinline__ void load_q(const unsigned char* codes, int so, bool e4m3, int j, float2 (&v)[H]) const {
    if constexpr (ALN) {
      const int c = c0 + j * 32;
      const float s = ckpt_scale(codes[so + (c * VEC) / kCkptGroup]);
      if constexpr (VEC == 8) {
        const uint2 u = reinterpret_cast<const uint2*>(codes)[c];
        if (e4m3) {
          ckpt_decode4(u.x, s, true, v[0], v[1]);
          ckpt_decode4(u.y, s, true, v[H - 2], v[H - 1]);
        } else {
          ckpt_decode4(u.x, s, false, v[0], v[1]);
          ckpt_decode4(u.y, s, false, v[H - 2], v[H - 1]);
        }
      } else {
        ckpt_decode4(reinterpret_cast<const uint32_t*>(codes)[c], s, e4m3, v[0], v[1]);
      }
    } else {
      // a warp's 32 columns of one k are a group; codes in pairs
      const unsigned char* q = codes + c0 + j * VEC * 32;
      const unsigned char* qs = codes + so + c0 / kCkptGroup + j * VEC;
      uint32_t u[VEC], e[VEC];
      if (whole(j)) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) { u[k] = q[k * 32]; e[k] = qs[k]; }
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const bool in = col(j, k) < NL;
          u[k] = in ? q[k * 32] : 0u;
          e[k] = in ? qs[k] : 1u;
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h)
        v[h] = fmul2(ckpt_pair(u[2 * h], u[2 * h + 1], e4m3),
                     make_float2(ckpt_scale(e[2 * h]), ckpt_scale(e[2 * h + 1])));
    }
  }
  // `at`: this thread's first chunk (column) of the row in global memory
  __device__ __forceinline__ void store(char* at, int j, const float2 (&v)[H]) const {
    if constexpr (ALN) {
      st_global_cs16(at + j * 512, P::pack(v));
    } else {
      T* q = reinterpret_cast<T*>(at) + j * VEC * 32;
      if (whole(j)) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) q[k * 32] = from_f<T>((k & 1) ? v[k / 2].y : v[k / 2].x);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (col(j, k) < NL) q[k * 32] = from_f<T>((k & 1) ? v[k / 2].y : v[k / 2].x);
      }
    }
  }
  // Encode chunk j into a checkpoint row; `codes`: this thread's first code,
  // `scale`: from there to its first scale.  Called by every thread of the warp
  // (the group's largest value travels between lanes); ok: chunk exists.
  __device__ __forceinline__ void encode(char* codes, int scale, bool e4m3, int j, const float2 (&v)[H],
                                         bool ok) const {
    if constexpr (ALN) {
      float am = 0.f;
      if (ok) {
#pragma unroll
        for (int h = 0; h < H; ++h) am = max_abs3(am, v[h].x, v[h].y);
      }
      constexpr int LANES = kCkptGroup / VEC;   // lanes that share a group
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (!ok) return;
      const uint32_t b = ckpt_scale_byte(__float_as_uint(am), e4m3);
      const float2 inv = f2s(ckpt_inv_scale(b));
      float2 u[H];
#pragma unroll
      for (int h = 0; h < H; ++h) u[h] = fmul2(v[h], inv);
      uint32_t w[VEC / 4];
      if (e4m3) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = ckpt_encode4(u[2 * i], u[2 * i + 1], true);
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = ckpt_encode4(u[2 * i], u[2 * i + 1], false);
      }
      if constexpr (VEC == 8) reinterpret_cast<uint2*>(codes)[j * 32] = make_uint2(w[0], w[VEC / 4 - 1]);
      else reinterpret_cast<uint32_t*>(codes)[j * 32] = w[0];
      if ((c0 & (LANES - 1)) == 0) codes[scale + j * (32 / LANES)] = (char)b;
    } else {
      // a warp's lanes hold 32 consecutive columns of one k: a group
      uint32_t e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float x = (k & 1) ? v[k / 2].y : v[k / 2].x;
        e[k] = ckpt_scale_byte(
            __reduce_max_sync(0xffffffffu, col(j, k) < NL ? __float_as_uint(x) & 0x7fffffffu : 0u), e4m3);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t u = ckpt_encode2(
            fmul2(v[h], make_float2(ckpt_inv_scale(e[2 * h]), ckpt_inv_scale(e[2 * h + 1]))), e4m3);
        if (col(j, 2 * h) < NL) codes[(j * VEC + 2 * h) * 32] = (char)u;
        if (col(j, 2 * h + 1) < NL) codes[(j * VEC + 2 * h + 1) * 32] = (char)(u >> 8);
      }
      if ((c0 & 31) == 0) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (col(j, k) < NL) codes[scale + j * VEC + k] = (char)e[k];
      }
    }
  }
  // Chunk j of a per-column vector, `base` its first column of the slice (0 beyond
  // the slice).  Aligned form: on 16 bytes.
  __device__ __forceinline__ void columns(const char* base, int code, int j, float2 (&v)[H]) const {
#pragma unroll
    for (int h = 0; h < H; ++h) v[h] = f2s(0.f);
    if (!has(j)) return;
    if constexpr (ALN) {
      const int c = c0 + j * 32;
      if (code == NORM_F32) {
#pragma unroll
        for (int h = 0; h < H; h += 2) {
          const float4 t = reinterpret_cast<const float4*>(base)[c * (VEC / 4) + h / 2];
          v[h] = make_float2(t.x, t.y);
          v[h + 1] = make_float2(t.z, t.w);
        }
      } else if constexpr (VEC == 8) {   // (16-bit vectors come with 16-bit rows)
        const uint4 u = reinterpret_cast<const uint4*>(base)[c];
        if (code == NORM_F16) Pack16<__half>::unpack(u, v);
        else Pack16<__nv_bfloat16>::unpack(u, v);
      }
    } else {
      // (one test of the type, then the loads side by side)
      if (code == NORM_F32) single<float>(base, j, v);
      else if (code == NORM_F16) single<__half>(base, j, v);
      else single<__nv_bfloat16>(base, j, v);
    }
  }
  template <class W>
  __device__ __forceinline__ void single(const char* base, int j, float2 (&v)[H]) const {
    const W* q = reinterpret_cast<const W*>(base) + c0 + j * VEC * 32;
    W t[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) t[k] = valid(j, k) ? q[k * 32] : from_f<W>(0.f);
#pragma unroll
    for (int h = 0; h < H; ++h) v[h] = make_float2(to_f(t[2 * h]), to_f(t[2 * h + 1]));
  }
  // Chunk j to a per-column vector of any type.
  __device__ __forceinline__ void store_columns(char* base, int code, int j, const float2 (&v)[H]) const {
    if constexpr (ALN) {
      const int c = c0 + j * 32;
      if (code == NORM_F32) {
#pragma unroll
        for (int h = 0; h < H; h += 2)
          reinterpret_cast<float4*>(base)[c * (VEC / 4) + h / 2] = make_float4(v[h].x, v[h].y, v[h + 1].x, v[h + 1].y);
      } else if constexpr (VEC == 8) {
        reinterpret_cast<uint4*>(base)[c] = code == NORM_F16 ? Pack16<__half>::pack(v) : Pack16<__nv_bfloat16>::pack(v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (valid(j, k)) st_code(base, code, col(j, k), (k & 1) ? v[k / 2].y : v[k / 2].x);
    }
  }
  // Chunk j of an FP32 partial row: out[col] = v (add: += v)
  __device__ __forceinline__ void partial(float* out, int j, const float2 (&v)[H], bool add) const {
    if constexpr (ALN) {
      if (!has(j)) return;
      float4* q = reinterpret_cast<float4*>(out + col(j, 0));
#pragma unroll
      for (int h = 0; h < H; h += 2) {
        float4 t = make_float4(v[h].x, v[h].y, v[h + 1].x, v[h + 1].y);
        if (add) {
          const float4 o = q[h / 2];
          t = make_float4(fadd(o.x, t.x), fadd(o.y, t.y), fadd(o.z, t.z), fadd(o.w, t.w));
        }
        q[h / 2] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int c = col(j, k);
        const float x = (k & 1) ? v[k / 2].y : v[k / 2].x;
        if (c < NL) out[c] = add ? fadd(out[c], x) : x;
      }
    }
  }
};

// Sum over the warp of up to four values at once: the first two butterfly steps
// hand half of the values to the other half of the lanes, so four values take 6
// shuffles in place of 20.  The total of value i is then with lanes 8 i .. 8 i + 7
// (two values: 16 i .. 16 i + 15; one: all lanes).
template <int NV>
__device__ __forceinline__ float warp_sum_spread(const float (&v)[NV], int lane) {
  float a;
  int o;
  if constexpr (NV >= 3) {
    const bool up = lane & 16, up2 = lane & 8;
    const float v3 = NV > 3 ? v[NV > 3 ? 3 : 0] : 0.f;
    const float k0 = fadd(up ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16));
    const float k1 = fadd(up ? v3 : v[1], __shfl_xor_sync(0xffffffffu, up ? v[1] : v3, 16));
    a = fadd(up2 ? k1 : k0, __shfl_xor_sync(0xffffffffu, up2 ? k0 : k1, 8));
    o = 4;
  } else if constexpr (NV == 2) {
    const bool up = lane & 16;
    a = fadd(up ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16));
    o = 8;
  } else {
    a = fadd(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
    o = 8;
  }
  for (; o > 0; o >>= 1) a = fadd(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Sums over the row: over the CTA (within the warps, then over the warps' sums;
// two banks used in turn, one barrier a call), then over the cluster's CTAs in
// rank order.  Every thread ends with the same bits.
template <bool CL>
struct RowSum {
  float* red;        // [2][16][4], zeroed: entries beyond the CTA's warps stay zero
  float4* xch;       // [2][8]
  uint64_t* xbar;    // [2]
  int* abort_flag;   // [2]
  int* status;
  int tid = 0, bank = 0, xn = 0, steps = 0, ncl = 1, crank = 0;

  template <int NV>
  __device__ __forceinline__ void operator()(float (&v)[NV], int next_fl) {
    static_assert(NV <= 4, "a float4 a warp");
    constexpr int SPAN = NV >= 3 ? 8 : NV == 2 ? 16 : 32;   // lanes that hold one value's total
    const int warp = tid >> 5, lane = tid & 31;
    const float a = warp_sum_spread<NV>(v, lane);
    float* r = red + bank * 64;
    if ((lane & (SPAN - 1)) == 0 && lane / SPAN < NV) r[warp * 4 + lane / SPAN] = a;
    __syncthreads();
    const float4 t = reinterpret_cast<const float4*>(r)[lane & (steps - 1)];
    v[0] = t.x;
    if constexpr (NV > 1) v[1] = t.y;
    if constexpr (NV > 2) v[2] = t.z;
    for (int o = steps >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = fadd(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
    bank ^= 1;
    if constexpr (CL) {
      if (ncl > 1) exchange(v, next_fl);
    }
  }
  // Thread 0 stores the CTA's sums into every peer, completing on the peer's
  // mbarrier.  Slots alternate; a peer sends its next values only after it has
  // received these, and a CTA only after all its threads have passed the
  // barrier above, so a slot is never overwritten while it is read.  A wait
  // that runs out raises the abort flag of the next row.
  template <int NV>
  __device__ __forceinline__ void exchange(float (&v)[NV], int next_fl) {
    constexpr int NS = NV <= 2 ? 2 : 4;
    const int slot = xn & 1;
    const uint32_t ph = (uint32_t)((xn >> 1) & 1);
    ++xn;
    if (tid == 0) {
      mbar_arrive_expect_tx(&xbar[slot], (uint32_t)((ncl - 1) * NS * 4));
      const uint32_t mine = smem_addr(&xch[slot * 8 + crank]);
      const uint32_t bar = smem_addr(&xbar[slot]);
      for (int q = 0; q < ncl; ++q) {
        if (q == crank) continue;
        const uint32_t dst = map_shared_rank(mine, q), rb = map_shared_rank(bar, q);
        st_async_f32x2(dst, v[0], NV > 1 ? v[NV > 1] : 0.f, rb);
        if constexpr (NS == 4) st_async_f32x2(dst + 8, v[NV > 2 ? 2 : 0], 0.f, rb);
      }
    }
    if (!mbar_wait_cluster_bounded(&xbar[slot], ph)) {
      atomicOr(status, STATUS_WAIT_TIMEOUT);
      abort_flag[next_fl] = 1;
    }
    float t[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) t[i] = 0.f;
    for (int q = 0; q < ncl; ++q) {
      const float4 o = xch[slot * 8 + q];
      const float w[3] = {o.x, o.y, o.z};
#pragma unroll
      for (int i = 0; i < NV; ++i) t[i] = fadd(t[i], q == crank ? v[i] : w[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = t[i];
  }
};

// One bulk copy of every row: where its slice starts in the current row (moved
// on by `step` with every row), the slice's bytes, its place in a stage, and the
// matrix's extent (general form).  A gate row serves R rows: `rem` counts the row
// within them, `rem_step` is what a step adds, and a carry moves on by `carry`.
struct CopySlot {
  const char* src;
  int64_t step;
  const char* lo;
  const char* hi;
  int64_t rem, rem_step, carry;
  uint32_t len, dst;
};
constexpr int kCopySlots = 8;

// What both kernels set up: the CTA's slice, its rows (every G-th, or a
// contiguous range: seg), the ring and its copies.  Thread `s` of the first warp
// makes slot s, so that a row's copies are issued side by side.
#define GB300NORM_BLOCK_PROLOGUE(QX)                                                                                   \
  using IO = RowIO<T, NPT, ALN>;                                                                                       \
  constexpr int VEC = IO::VEC;                                                                                         \
  constexpr int H = IO::H;                                                                                             \
  extern __shared__ __align__(128) unsigned char smem[];                                                               \
  __shared__ __align__(16) float red[2][16][4];                                                                        \
  __shared__ float4 xch[2][8];                                                                                         \
  __shared__ __align__(8) uint64_t xbar[2];                                                                            \
  __shared__ CopySlot slots[kCopySlots];                                                                               \
  __shared__ int abort_flag[2];                                                                                        \
  int tid;   /* read once: the compiler would read the special register again at every use */                          \
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));                                                                    \
  const int nt = blockDim.x, lane = tid & 31, warp = tid >> 5;                                                         \
  const int N = p.N;                                                                                                   \
  RowSum<CL> sum;                                                                                                      \
  sum.tid = tid;                                                                                                       \
  if constexpr (CL) {                                                                                                  \
    sum.ncl = (int)cluster_nctarank();                                                                                 \
    sum.crank = (int)cluster_ctarank();                                                                                \
  }                                                                                                                    \
  const int ncl = CL ? sum.ncl : 1, crank = CL ? sum.crank : 0;                                                        \
  IO io;                                                                                                               \
  io.place(warp, lane);                                                                                                \
  int col0;                                                                                                            \
  if constexpr (ALN) {                                                                                                 \
    io.nch = N / VEC / ncl;                                                                                            \
    io.NL = io.nch * VEC;                                                                                              \
    col0 = crank * io.NL;                                                                                              \
  } else {                                                                                                             \
    const int part = p.part;                                                                                           \
    col0 = crank * part;                                                                                               \
    io.NL = N - col0 < part ? N - col0 : part;                                                                         \
    io.nch = 0;                                                                                                        \
  }                                                                                                                    \
  sum.red = &red[0][0][0];                                                                                             \
  sum.xch = &xch[0][0];                                                                                                \
  sum.xbar = xbar;                                                                                                     \
  sum.abort_flag = abort_flag;                                                                                         \
  sum.status = p.status;                                                                                               \
  sum.steps = 1;                                                                                                       \
  while (sum.steps * 32 < nt) sum.steps *= 2;                                                                          \
  const int64_t G = gridDim.x / ncl;                                                                                   \
  const int64_t grp = blockIdx.x / ncl;                                                                                \
  const int64_t row0 = p.seg ? seg_begin(grp, p.M, G) : grp;                                                           \
  const int step = (int)p.row_step;                                                                                    \
  const int nrows = (int)(p.seg ? seg_begin(grp + 1, p.M, G) - row0 : (p.M - grp + G - 1) / G);                        \
  const float inv_n = 1.0f / (float)N;                                                                                 \
  const bool e4m3 = p.fmt == NORM_SAVED_E4M3;                                                                          \
  const int scale_off = (int)ckpt_scale_off(N);                                                                        \
  const int stage_so = (io.NL + 15) / 16 * 16;   /* a staged checkpoint slice's scales */                              \
  const int64_t cb = (int64_t)col0 * (int64_t)sizeof(T);                                                               \
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                                                                  \
  unsigned char* stages = smem + kBlockHeader;                                                                         \
  for (int i = tid; i < 128; i += nt) (&red[0][0][0])[i] = 0.f;                                                        \
  const uint64_t pol = l2_policy_evict_first();                                                                        \
  int issued = 0, istage = 0;                                                                                          \
  /* first warp: copies of rows issued .. limit-1 */                                                                   \
  auto issue_to = [&](int limit) {                                                                                     \
    if (limit > nrows - p.hold_last) limit = nrows - p.hold_last;                                                      \
    _Pragma("unroll 1") for (; issued < limit; ++issued) {                                                             \
      block_issue<ALN>(slots, p, stages + (size_t)istage * p.stage_bytes, &bars[istage], pol, lane);                   \
      if (++istage == S) istage = 0;                                                                                   \
    }                                                                                                                  \
  };                                                                                                                   \
  if (warp == 0) {                                                                                                     \
    if (lane < kCopySlots) slots[lane] = block_slot<T, QX, ALN>(p, lane, row0, step, col0, io.NL, scale_off);          \
    if (lane == 0) {                                                                                                   \
      _Pragma("unroll 1") for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);                                          \
      if constexpr (CL) { mbar_init(&xbar[0], 1); mbar_init(&xbar[1], 1); }                                            \
      fence_mbar_init();                                                                                               \
      abort_flag[0] = 0;                                                                                               \
      abort_flag[1] = 0;                                                                                               \
    }                                                                                                                  \
    __syncwarp();                                                                                                      \
  }                                                                                                                    \
  grid_dependency_wait();   /* nothing above reads what an earlier kernel wrote */                                     \
  if (warp == 0) issue_to(S);

// Slot i: the five streams, then the scales of the checkpoint streams.
template <class T, bool QX, bool ALN>
__device__ __forceinline__ CopySlot block_slot(const BlockParams& p, int i, int64_t row0, int64_t step, int col0,
                                               int NL, int scale_off) {
  CopySlot c = {};
  const int s = i < kBlockStreams ? i : i == kBlockStreams ? SX : SH;
  const bool q = QX && (s == SX || s == SH);
  if (i > kBlockStreams + 1 || !p.in[s] || (i >= kBlockStreams && !q)) return c;
  c.src = p.in[s] + row0 * p.in_stride[s];
  c.step = step * p.in_stride[s];
  c.dst = p.soff[s];
  c.hi = reinterpret_cast<const char*>(~(uintptr_t)0);
  if (q) {
    // codes and scales: slices padded to 16 bytes, always aligned
    const uint32_t nc = (uint32_t)((NL + 15) / 16 * 16);
    if (i < kBlockStreams) {
      c.src += col0;
      c.len = nc;
    } else {
      c.src += scale_off + col0 / kCkptGroup;
      c.len = (uint32_t)((NL + 511) / 512 * 16);
      c.dst += nc;
    }
    return c;
  }
  const int64_t off = (int64_t)col0 * (int64_t)sizeof(T);
  c.src += off;
  c.len = (uint32_t)NL * (uint32_t)sizeof(T);
  if (!ALN) {
    c.lo = p.in[s];
    c.hi = p.in[s] + ((s == SG ? p.n_gates : p.M) - 1) * p.in_stride[s] + (int64_t)p.N * (int64_t)sizeof(T);
  }
  if (s == SG && p.R > 1) {
    c.src = p.in[s] + off + row0 / p.R * p.in_stride[s];
    c.step = step / p.R * p.in_stride[s];
    c.rem = row0 % p.R;
    c.rem_step = step % p.R;
    c.carry = p.in_stride[s];
  }
  return c;
}

// One row's copies into stage `dst` (the first warp).
template <bool ALN>
__device__ __forceinline__ void block_issue(CopySlot* slots, const BlockParams& p, unsigned char* dst, uint64_t* bar,
                                            uint64_t pol, int lane) {
  uint32_t len = 0, to = 0;
  const char* src = nullptr;
  if (lane < kCopySlots) {
    CopySlot& c = slots[lane];
    src = c.src;
    len = c.len;
    to = c.dst;
    const char* next = src + c.step;
    if (c.carry) {
      int64_t rem = c.rem + c.rem_step;
      if (rem >= p.R) {
        rem -= p.R;
        next += c.carry;
      }
      c.rem = rem;
    }
    c.src = next;
    if (!ALN && len) {
      // rounded out to 16 bytes where that stays within the matrix, else in
      uintptr_t a = reinterpret_cast<uintptr_t>(src), b = a + len;
      const uintptr_t base = a & ~(uintptr_t)15;
      const uintptr_t lo = base >= reinterpret_cast<uintptr_t>(c.lo) ? base : (a + 15) & ~(uintptr_t)15;
      const uintptr_t up = (b + 15) & ~(uintptr_t)15;
      const uintptr_t hi = up <= reinterpret_cast<uintptr_t>(c.hi) ? up : b & ~(uintptr_t)15;
      len = hi > lo ? (uint32_t)(hi - lo) : 0u;
      to += (uint32_t)(lo - base);
      src = reinterpret_cast<const char*>(lo);
    }
  }
  const uint32_t bytes = ALN ? p.stage_bytes : __reduce_add_sync(0xffffffffu, len);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
  __syncwarp();
  if (len) bulk_g2s(dst + to, src, len, bar, pol);
}

// General form: whether a row's copies, rounded out to 16 bytes, stay within
// every streamed matrix.
__device__ __forceinline__ bool row_is_clean(const BlockParams& p, int64_t row, int64_t rows) {
  return row * p.min_stride >= 15 && (rows - 1 - row) * p.min_stride >= 15;
}

// mbar_wait_bounded (common.cuh) in few instructions: false once kWaitLimitNs
// have passed.
__device__ __forceinline__ bool block_wait(uint64_t* bar, uint32_t parity, uint64_t deadline = 0) {
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t now = global_timer_ns();
    if (deadline == 0) deadline = now + kWaitLimitNs;
    if (now > deadline) return false;
  }
}

// General form, a row whose copies were rounded in: the slice's elements outside
// them (at most 15 bytes at either end) from global memory into the stage.
// `at`: the slice's start there.  Called by the whole CTA.
template <class T>
__device__ __forceinline__ void block_edges(unsigned char* at, const char* src, int NL) {
  const T* g = reinterpret_cast<const T*>(src);
  T* s = reinterpret_cast<T*>(at);
  constexpr int E = 16 / (int)sizeof(T);
  const int head = (int)(((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / sizeof(T));
  const int tail = (int)((reinterpret_cast<uintptr_t>(src + (int64_t)NL * (int64_t)sizeof(T)) & 15) / sizeof(T));
  const int i = (int)threadIdx.x & 15;   // lanes 0 .. E-1: head, 16 - E ..: tail
  if (threadIdx.x < E) {
    if (i < head && i < NL) s[i] = g[i];
  } else if (threadIdx.x >= 16 && threadIdx.x < 16 + E) {
    const int c = NL - tail + i;
    if (i < tail && c >= 0) s[c] = g[c];
  }
}

// What a wait that ran out leaves to do: the copies still in flight into this
// CTA's shared memory (rows k .. issued-1, the first warp's count).
__device__ __forceinline__ void block_drain(uint64_t* bars, int S, int k, int issued, int s, uint32_t phase) {
  const uint64_t deadline = global_timer_ns() + kWaitLimitNs;
#pragma unroll 1
  for (; k < issued; ++k) {
    if (!block_wait(&bars[s], phase, deadline)) break;
    if (++s == S) { s = 0; phase ^= 1u; }
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <class T, int FORM, bool GROW, bool Q8, int ALT, bool ALN, bool CL>
__global__ void __launch_bounds__(fwd_cta(FORM, Q8, ALT, ALN).threads, fwd_cta(FORM, Q8, ALT, ALN).ctas)
    block_fwd_kernel(const BlockParams p, const int S) {
  constexpr int NPT = fwd_cta(FORM, Q8, ALT, ALN).cols * (int)sizeof(T) / 16;
  GB300NORM_BLOCK_PROLOGUE(false)
  constexpr bool LN = FORM == kLn;
  const bool post = FORM == kDynamic ? p.post != 0 : FORM == kBoth || FORM == kPost;
  const bool pre = FORM == kDynamic ? p.pre != 0 : FORM != kPost;
  // per-column values: cv = b g W1' (the bias for LayerNorm), w2 = W2'
  constexpr bool C = FORM != kNorm;
  constexpr int NC = C ? NPT : 1;
  float2 cv[NC][H], w2[NPT][H];
  auto slice = [&](const void* v, int code) { return static_cast<const char*>(v) + (int64_t)col0 * code_size(code); };
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    float2 t[H];
    if constexpr (LN) {
#pragma unroll
      for (int h = 0; h < H; ++h) cv[j][h] = f2s(0.f);
      if (p.bias) io.columns(slice(p.bias, p.w_code), p.w_code, j, cv[j]);
    } else if constexpr (C) {
#pragma unroll
      for (int h = 0; h < H; ++h) cv[j][h] = f2s(p.beta);
      if (p.w1) {
        io.columns(slice(p.w1, p.w_code), p.w_code, j, t);
#pragma unroll
        for (int h = 0; h < H; ++h) cv[j][h] = fmul2(fadd2(t[h], f2s(p.offset)), cv[j][h]);
      }
      if (p.gate) {
        io.columns(slice(p.gate, p.gate_code), p.gate_code, j, t);
#pragma unroll
        for (int h = 0; h < H; ++h) cv[j][h] = fmul2(cv[j][h], t[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) w2[j][h] = f2s(0.f);
    if (p.w2) {
      io.columns(slice(p.w2, p.w_code), p.w_code, j, t);
#pragma unroll
      for (int h = 0; h < H; ++h) w2[j][h] = fadd2(t[h], f2s(p.offset));
    }
  }
  if constexpr (CL) cluster_barrier();
  else __syncthreads();

  const bool has_r = p.in[SR] != nullptr;
  const bool want_h = p.out_a != nullptr;
  // where this thread's columns of a row go, moved on with the rows
  char* hrow = p.out_a + row0 * p.a_stride + cb + io.at();
  char* yrow = p.out_b + row0 * p.b_stride + cb + io.at();
  // this thread's first code in a checkpoint row, and from there to its scale
  const int qcol = col0 + io.col(0, 0);
  const int64_t qoff = row0 * p.q_stride + qcol;
  char* xq = p.xq + qoff;
  char* hq = p.hq + qoff;
  const int qscale = scale_off + qcol / kCkptGroup - qcol;
  const bool keep_x = Q8 && p.xq != nullptr, keep_h = Q8 && p.hq != nullptr;
  int64_t row = row0;
  bool aborted = false;
  int k = 0, s = 0;
  uint32_t phase = 0;
  const unsigned char* stage = stages;
  for (; k < nrows; ++k) {
    const int fl = k & 1;
    if (!block_wait(&bars[s], phase)) {
      atomicOr(p.status, STATUS_WAIT_TIMEOUT);
      abort_flag[fl] = 1;
    }
    auto from = [&](int q) { return p.in[q] + (q == SG ? row / p.R : row) * p.in_stride[q] + cb; };
    // a streamed slice in the stage (general form: at its own offset from 16 bytes)
    auto src = [&](int q) -> const unsigned char* {
      if constexpr (ALN) return stage + p.soff[q];
      return stage + p.soff[q] + ((uint32_t)(uintptr_t)from(q) & 15u);
    };
    if constexpr (!ALN) {
      if (!(row_is_clean(p, row, p.M) && (!GROW || row_is_clean(p, row / p.R, p.n_gates)))) {
        for (int q = 0; q < kBlockStreams; ++q)
          if (p.in[q]) block_edges<T>(const_cast<unsigned char*>(src(q)), from(q), io.NL);
        __syncthreads();
      }
    }
    const unsigned char* gx = src(SX);
    float2 hv[NPT][H];
    if constexpr (LN) {
      float2 acc[H];
#pragma unroll
      for (int h = 0; h < H; ++h) acc[h] = f2s(0.f);
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
#pragma unroll
        for (int h = 0; h < H; ++h) hv[j][h] = f2s(0.f);
        if (!io.has(j)) continue;
        io.load(gx, j, hv[j]);
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = fadd2(acc[h], hv[j][h]);
      }
      float a[1] = {tree_sum<H>(acc)};
      sum(a, fl ^ 1);
      if (abort_flag[fl]) { aborted = true; break; }
      if (warp == 0) issue_to(k + 1 + S);   // the row is in registers: its stage is free
      const float mean = div_n(a[0], inv_n);
#pragma unroll
      for (int h = 0; h < H; ++h) acc[h] = f2s(0.f);
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        if (io.has(j)) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            hv[j][h] = fadd2(hv[j][h], f2s(-mean));
            if constexpr (!ALN)   // (columns beyond the row count nothing)
              hv[j][h] = make_float2(io.valid(j, 2 * h) ? hv[j][h].x : 0.f, io.valid(j, 2 * h + 1) ? hv[j][h].y : 0.f);
            acc[h] = ffma2(hv[j][h], hv[j][h], acc[h]);
          }
        }
        // the checkpoint is of x - mean, which is all the backward uses of x
        if constexpr (Q8) io.encode(hq, qscale, e4m3, j, hv[j], io.has(j));
      }
      float q[1] = {tree_sum<H>(acc)};
      sum(q, fl ^ 1);
      const float rstd = inv_rms(div_n(q[0], inv_n), p.eps);
      if (tid == 0 && crank == 0) {
        if (p.mean_out) p.mean_out[row] = mean;
        if (p.rs2_out) p.rs2_out[row] = rstd;
      }
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        if (!io.has(j)) continue;
        float2 o[H];
#pragma unroll
        for (int h = 0; h < H; ++h) o[h] = ffma2(fmul2(hv[j][h], f2s(rstd)), w2[j][h], cv[j][h]);
        io.store(yrow, j, o);
      }
    } else {
      float rs1 = 1.f;
      if (post) {
        float2 acc[H];
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = f2s(0.f);
#pragma unroll
        for (int j = 0; j < NPT; ++j) {
          const bool ok = io.has(j);
          float2 x[H];
          if (ok) {
            io.load(gx, j, x);
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = ffma2(x[h], x[h], acc[h]);
          }
          if constexpr (Q8) {
            if (keep_x) io.encode(xq, qscale, e4m3, j, x, ok);
          }
        }
        float a[1] = {tree_sum<H>(acc)};
        sum(a, fl ^ 1);
        if (abort_flag[fl]) { aborted = true; break; }
        // (without a second norm this is the row's only barrier: it says that
        // the row before is done)
        if (warp == 0 && !pre) issue_to(k + S);
        rs1 = inv_rms(div_n(a[0], inv_n), p.eps);
        if (tid == 0 && crank == 0 && p.rs1_out) p.rs1_out[row] = rs1;
      }
      const unsigned char* gr = src(has_r ? SR : SX);
      const unsigned char* gg = src(GROW ? SG : SX);
      float2 acc[H];
#pragma unroll
      for (int h = 0; h < H; ++h) acc[h] = f2s(0.f);
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        const bool ok = io.has(j);
#pragma unroll
        for (int h = 0; h < H; ++h) hv[j][h] = f2s(0.f);
        float2 x[H];
        if (ok) {
          float2 t[H];
          io.load(gx, j, x);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            if constexpr (C) hv[j][h] = post ? fmul2(fmul2(x[h], f2s(rs1)), cv[j][h]) : fmul2(x[h], cv[j][h]);
            else hv[j][h] = x[h];
          }
          if constexpr (GROW) {
            io.load(gg, j, t);
#pragma unroll
            for (int h = 0; h < H; ++h) hv[j][h] = fmul2(hv[j][h], t[h]);
          }
          if (has_r) {
            io.load(gr, j, t);
#pragma unroll
            for (int h = 0; h < H; ++h) hv[j][h] = C ? ffma2(t[h], f2s(p.alpha), hv[j][h]) : fadd2(t[h], hv[j][h]);
          }
          if (want_h) io.store(hrow, j, hv[j]);
          if (pre) {
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = ffma2(hv[j][h], hv[j][h], acc[h]);
          }
        }
        if constexpr (Q8) {
          if (keep_h) io.encode(hq, qscale, e4m3, j, hv[j], ok);
          if (!post && keep_x) io.encode(xq, qscale, e4m3, j, x, ok);
        }
      }
      if (pre) {
        float a[1] = {tree_sum<H>(acc)};
        sum(a, fl ^ 1);
        if (abort_flag[fl]) { aborted = true; break; }
        if (warp == 0) issue_to(k + 1 + S);   // h is in registers: the row's stage is free
        const float rs2 = inv_rms(div_n(a[0], inv_n), p.eps);
        if (tid == 0 && crank == 0 && p.rs2_out) p.rs2_out[row] = rs2;
#pragma unroll
        for (int j = 0; j < NPT; ++j) {
          if (!io.has(j)) continue;
          float2 o[H];
#pragma unroll
          for (int h = 0; h < H; ++h) o[h] = fmul2(fmul2(hv[j][h], f2s(rs2)), w2[j][h]);
          io.store(yrow, j, o);
        }
      }
    }
    row += p.row_step;
    hrow += p.a_step;
    yrow += p.b_step;
    if constexpr (Q8) { xq += p.q_step; hq += p.q_step; }
    stage += p.stage_bytes;
    if (++s == S) { s = 0; phase ^= 1u; stage = stages; }
  }
  grid_launch_dependents();
  if (aborted && warp == 0) block_drain(bars, S, k, issued, s, phase);
  if constexpr (CL) cluster_barrier();   // peers may still store into this CTA's shared memory
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// Row groups write partial rows: ws1 (dw1), ws2 (dw2), and for a gate with
// fewer rows than M the sums b A of its rows.  With one gate row every group
// writes its sum to ws_head.  With more (seg) a group owns a contiguous range
// of rows; when the gate row changes it adds g b A to its dw1 row and hands
// b A on: straight to the gate's gradient where all of that gate row's rows
// are the group's own, else to ws_head (its first gate row) or ws_tail (its
// last), for launch_block_reduce.
template <class T, int FORM, int GATE, bool Q8, bool ACC, int ALT, bool ALN, bool CL>
__global__ void __launch_bounds__(bwd_cta(FORM, ALT, ALN).threads, bwd_cta(FORM, ALT, ALN).ctas)
    block_bwd_kernel(const BlockParams p, const int S) {
  constexpr bool GROW = GATE == kStreamed, SEG = GATE == kSegments;
  constexpr int NPT = bwd_cta(FORM, ALT, ALN).cols * (int)sizeof(T) / 16;
  GB300NORM_BLOCK_PROLOGUE(Q8)
  constexpr bool LN = FORM == kLn;
  const bool post = FORM == kDynamic ? p.post != 0 : FORM == kBoth || FORM == kPost;
  const bool pre = FORM == kDynamic ? p.pre != 0 : FORM != kPost;
  constexpr bool X = FORM != kLn && FORM != kNorm;   // x, its norm and gate may be there
  constexpr int NC = X ? NPT : 1;
  float2 cv[NC][H], w2[NPT][H];
  // one norm's two input rows stay in registers from the sums to the outputs (a
  // second load and decoding saved)
  constexpr bool KEEP = ALN && (FORM == kLn || (one_norm(FORM) && ALT != 1));
  constexpr int NK = KEEP ? NPT : 1;
  constexpr int NA = ACC ? NPT : 1;
  constexpr int NA1 = ACC && FORM != kNorm ? NPT : 1;
  float2 acc1[NA1][H], acc2[NA][H];   // A (dB for LayerNorm), dw2
#pragma unroll
  for (int j = 0; j < NA; ++j)
#pragma unroll
    for (int h = 0; h < H; ++h) { acc1[j < NA1 ? j : 0][h] = f2s(0.f); acc2[j][h] = f2s(0.f); }
  auto slice = [&](const void* v, int code) { return static_cast<const char*>(v) + (int64_t)col0 * code_size(code); };
  // this slice of gate row q
  auto gate_row = [&](int64_t q) { return slice(p.gate, p.gate_code) + q * p.gate_stride * code_size(p.gate_code); };
  // cv = b W1' g of gate row q (without the streamed gate)
  auto form_c = [&](int64_t q) {
    if constexpr (X) {
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        float2 t[H];
#pragma unroll
        for (int h = 0; h < H; ++h) cv[j][h] = f2s(p.beta);
        if (p.w1) {
          io.columns(slice(p.w1, p.w_code), p.w_code, j, t);
#pragma unroll
          for (int h = 0; h < H; ++h) cv[j][h] = fmul2(fadd2(t[h], f2s(p.offset)), cv[j][h]);
        }
        if (!GROW && p.gate) {
          io.columns(gate_row(q), p.gate_code, j, t);
#pragma unroll
          for (int h = 0; h < H; ++h) cv[j][h] = fmul2(cv[j][h], t[h]);
        }
      }
    }
  };
  const int64_t q_first = SEG ? row0 / p.R : 0;
  int64_t q_now = q_first;   // the gate row in cv
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
#pragma unroll
    for (int h = 0; h < H; ++h) w2[j][h] = f2s(0.f);
    if (p.w2) {
      float2 t[H];
      io.columns(slice(p.w2, p.w_code), p.w_code, j, t);
#pragma unroll
      for (int h = 0; h < H; ++h) w2[j][h] = fadd2(t[h], f2s(p.offset));
    }
  }
  if constexpr (CL) cluster_barrier();
  else __syncthreads();

  // acc1 (of gate row q_now, whose rows end before row q_end) to the partial
  // rows; cleared
  auto flush = [&](int64_t q_end) {
    if constexpr (ACC && X) {
      // all of this gate row's rows are this group's own
      const bool own = SEG ? q_now * p.R >= row0 && q_end <= row0 + nrows : G == 1;
      const bool want_dg = !GROW && p.dg != nullptr;
      float* seg = q_now == q_first ? p.ws_head : p.ws_tail;
#pragma unroll
      for (int j = 0; j < NA1; ++j) {
        float2 t[H], a[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
          a[h] = fmul2(acc1[j][h], f2s(p.beta));
          acc1[j][h] = f2s(0.f);
        }
        if (want_dg) {
          if (own) {
            float2 d[H];
#pragma unroll
            for (int h = 0; h < H; ++h) d[h] = a[h];
            if (p.w1) {
              io.columns(slice(p.w1, p.w_code), p.w_code, j, t);
#pragma unroll
              for (int h = 0; h < H; ++h) d[h] = fmul2(fadd2(t[h], f2s(p.offset)), d[h]);
            }
            if (io.has(j))
              io.store_columns(p.dg + q_now * p.dg_stride + (int64_t)col0 * code_size(p.gate_code), p.gate_code, j, d);
          } else {
            io.partial(seg + grp * N + col0, j, a, false);
          }
        }
        if (p.ws1) {
          if (!GROW && p.gate) {
            io.columns(gate_row(q_now), p.gate_code, j, t);
#pragma unroll
            for (int h = 0; h < H; ++h) a[h] = fmul2(a[h], t[h]);
          }
          io.partial(p.ws1 + grp * N + col0, j, a, SEG && q_now != q_first);
        }
      }
    }
  };

  const bool has_dh = p.in[SR] != nullptr, has_x = p.in[SX] != nullptr;
  const bool want_dr = p.out_a != nullptr, want_dx = p.out_b != nullptr, want_dg = GROW && p.dg != nullptr;
  // row statistics, read one row ahead
  float rs1n = 1.f, rs2n = 0.f;
  if (post) rs1n = p.rs1[row0];
  if (pre) rs2n = p.rs2[row0];
  // where this thread's columns of a row go, moved on with the rows
  char* arow = p.out_a + row0 * p.a_stride + cb + io.at();
  char* brow = p.out_b + row0 * p.b_stride + cb + io.at();
  char* grow = p.dg + row0 * p.dg_stride + cb + io.at();
  int64_t row = row0;
  bool aborted = false;
  int k = 0, s = 0;
  uint32_t phase = 0;
  const unsigned char* stage = stages;
  // the rows of one gate row after another (all rows, without seg)
  for (; k < nrows && !aborted; q_now += SEG) {
    const int64_t q_end = SEG ? ((q_now + 1) * p.R < p.M ? (q_now + 1) * p.R : p.M) : p.M;
    const int k_end = SEG && q_end - row0 < nrows ? (int)(q_end - row0) : nrows;
    form_c(q_now);
    for (; k < k_end; ++k) {
      const int fl = k & 1;
      const float rs1 = rs1n, rs2 = rs2n;
      if (k + 1 < nrows) {
        if (post) rs1n = p.rs1[row + p.row_step];
        if (pre) rs2n = p.rs2[row + p.row_step];
      }
      if (!block_wait(&bars[s], phase)) {
        atomicOr(p.status, STATUS_WAIT_TIMEOUT);
        abort_flag[fl] = 1;
      }
      // a streamed slice in the stage (general form: rows of the activations' type
      // at their own offset from 16 bytes; a streamed gate has a row for each)
      auto from = [&](int q) { return p.in[q] + row * p.in_stride[q] + cb; };
      auto src = [&](int q) -> const unsigned char* {
        if (ALN || (Q8 && (q == SX || q == SH))) return stage + p.soff[q];
        return stage + p.soff[q] + ((uint32_t)(uintptr_t)from(q) & 15u);
      };
      if constexpr (!ALN) {
        if (!row_is_clean(p, row, p.M)) {
          for (int q = 0; q < kBlockStreams; ++q)
            if (p.in[q] && !(Q8 && (q == SX || q == SH)))
              block_edges<T>(const_cast<unsigned char*>(src(q)), from(q), io.NL);
          __syncthreads();
        }
      }
      const unsigned char *gx = src(SX), *gd = src(SR), *gy = src(SDY), *gh = src(SH), *gg = src(SG);
      auto load_x = [&](int j, float2 (&v)[H]) {
        if constexpr (Q8) io.load_q(gx, stage_so, e4m3, j, v);
        else io.load(gx, j, v);
      };
      auto load_h = [&](int j, float2 (&v)[H]) {
        if constexpr (Q8) io.load_q(gh, stage_so, e4m3, j, v);
        else io.load(gh, j, v);
      };
      // ---- the sums -------------------------------------------------------
      //  LN: sum g2 h, sum g2.  else: sum g2 h, sum (rs2 g2 + dh_out) C x,
      //  sum h C x (the last two with a first norm only)
      float2 kd[NK][H], kv[NK][H];   // (KEEP) dy and h, or dh_out and x
      float2 a0[H], a1[H], a2[H];
  #pragma unroll
      for (int h = 0; h < H; ++h) { a0[h] = f2s(0.f); a1[h] = f2s(0.f); a2[h] = f2s(0.f); }
  #pragma unroll
      for (int j = 0; j < NPT; ++j) {
        if (!io.has(j)) continue;
        float2 u[H], hh[H], t[H];
        if (pre) {
          io.load(gy, j, t);
          load_h(j, hh);
  #pragma unroll
          for (int h = 0; h < H; ++h) {
            u[h] = fmul2(t[h], w2[j][h]);
            a0[h] = ffma2(u[h], hh[h], a0[h]);
            if constexpr (KEEP) { kd[j][h] = t[h]; kv[j][h] = hh[h]; }
            if constexpr (LN) a1[h] = ffma2(t[h], w2[j][h], a1[h]);
          }
        }
        if (X && post) {
          if (has_dh) {
            io.load(gd, j, t);
  #pragma unroll
            for (int h = 0; h < H; ++h) {
              u[h] = pre ? ffma2(u[h], f2s(rs2), t[h]) : t[h];
              if constexpr (KEEP) kd[j][h] = t[h];
            }
          } else {
  #pragma unroll
            for (int h = 0; h < H; ++h) u[h] = fmul2(u[h], f2s(rs2));
          }
          load_x(j, t);
  #pragma unroll
          for (int h = 0; h < H; ++h) {
            if constexpr (KEEP) kv[j][h] = t[h];
            t[h] = fmul2(t[h], cv[X ? j : 0][h]);
          }
          if constexpr (GROW) {
            float2 g[H];
            io.load(gg, j, g);
  #pragma unroll
            for (int h = 0; h < H; ++h) t[h] = fmul2(t[h], g[h]);
          }
  #pragma unroll
          for (int h = 0; h < H; ++h) {
            a1[h] = ffma2(u[h], t[h], a1[h]);
            if (pre) a2[h] = ffma2(hh[h], t[h], a2[h]);
          }
        }
      }
      float s0 = 0.f, s1 = 0.f, s2 = 0.f;
      if constexpr (FORM == kLn) {
        float v[2] = {tree_sum<H>(a0), tree_sum<H>(a1)};
        sum(v, fl ^ 1);
        s0 = v[0]; s1 = v[1];
      } else if constexpr (FORM == kPre || FORM == kNorm) {
        float v[1] = {tree_sum<H>(a0)};
        sum(v, fl ^ 1);
        s0 = v[0];
      } else if constexpr (FORM == kPost) {
        float v[1] = {tree_sum<H>(a1)};
        sum(v, fl ^ 1);
        s1 = v[0];
      } else {
        float v[3] = {tree_sum<H>(a0), tree_sum<H>(a1), tree_sum<H>(a2)};
        sum(v, fl ^ 1);
        s0 = v[0]; s1 = v[1]; s2 = v[2];
      }
      if (abort_flag[fl]) { aborted = true; break; }
      if (warp == 0) issue_to(k + S);   // every thread is done with row k-1
      // dh = rs2 g2 + dh_out - kh h;  dx = rs1 (dh C - kx x)
      const float c2 = div_n(fmul(s0, rs2), inv_n);               // mean g2 xhat2
      const float kh = fmul(fmul(rs2, rs2), c2);
      const float kx = post ? fmul(fmul(rs1, rs1), div_n(ffma(-kh, s2, s1), inv_n)) : 0.f;
      const float nkx1 = -fmul(rs1, kx);
      const float nmg = LN ? -div_n(s1, inv_n) : 0.f;             // -mean g2
  #pragma unroll
      for (int j = 0; j < NPT; ++j) {
        if (!io.has(j)) continue;
        float2 dh[H], t[H];
        if (pre) {
          float2 hh[H];
          if constexpr (KEEP) {
  #pragma unroll
            for (int h = 0; h < H; ++h) { t[h] = kd[j][h]; hh[h] = kv[j][h]; }
          } else {
            io.load(gy, j, t);
            load_h(j, hh);
          }
          if constexpr (LN) {
            // dx = rs2 (dy W2' - mean g2 - xhat mean(g2 xhat))
  #pragma unroll
            for (int h = 0; h < H; ++h) {
              const float2 xh = fmul2(hh[h], f2s(rs2));
              dh[h] = fmul2(f2s(rs2), ffma2(xh, f2s(-c2), ffma2(t[h], w2[j][h], f2s(nmg))));
              if constexpr (ACC) {
                acc2[j][h] = ffma2(t[h], xh, acc2[j][h]);
                acc1[j][h] = fadd2(acc1[j][h], t[h]);
              }
            }
          } else {
            float2 d[H];
            if (has_dh) {
              io.load(gd, j, d);
            } else {
  #pragma unroll
              for (int h = 0; h < H; ++h) d[h] = f2s(0.f);
            }
  #pragma unroll
            for (int h = 0; h < H; ++h) {
              const float2 ty = fmul2(t[h], f2s(rs2));
              dh[h] = ffma2(hh[h], f2s(-kh), ffma2(ty, w2[j][h], d[h]));
              if constexpr (ACC) acc2[j][h] = ffma2(ty, hh[h], acc2[j][h]);
            }
          }
        } else if constexpr (KEEP) {
  #pragma unroll
          for (int h = 0; h < H; ++h) dh[h] = kd[j][h];
        } else {
          io.load(gd, j, dh);
        }
        if (want_dr) {
  #pragma unroll
          for (int h = 0; h < H; ++h) t[h] = X ? fmul2(dh[h], f2s(p.alpha)) : dh[h];
          io.store(arow, j, t);
        }
        if constexpr (X) {
          float2 x[H], g[H];
          // dh rs1 (and, streamed, times the gate)
          if (post) {
  #pragma unroll
            for (int h = 0; h < H; ++h) dh[h] = fmul2(dh[h], f2s(rs1));
          }
          if (has_x) {
            if constexpr (KEEP) {
  #pragma unroll
              for (int h = 0; h < H; ++h) x[h] = kv[j][h];
            } else {
              load_x(j, x);
            }
            if (want_dg) {
  #pragma unroll
              for (int h = 0; h < H; ++h) t[h] = fmul2(fmul2(dh[h], x[h]), cv[j][h]);
              io.store(grow, j, t);
            }
          }
          if constexpr (GROW) {
            io.load(gg, j, g);
  #pragma unroll
            for (int h = 0; h < H; ++h) dh[h] = fmul2(dh[h], g[h]);
          }
          if constexpr (ACC) {
            if (has_x) {
  #pragma unroll
              for (int h = 0; h < H; ++h) acc1[j][h] = ffma2(dh[h], x[h], acc1[j][h]);
            }
          }
          if (want_dx) {
  #pragma unroll
            for (int h = 0; h < H; ++h)
              t[h] = post ? ffma2(x[h], f2s(nkx1), fmul2(dh[h], cv[j][h])) : fmul2(dh[h], cv[j][h]);
            io.store(brow, j, t);
          }
        }
      }
      row += p.row_step;
      arow += p.a_step;
      brow += p.b_step;
      if constexpr (GROW) grow += p.dg_step;
      stage += p.stage_bytes;
      if (++s == S) { s = 0; phase ^= 1u; stage = stages; }
    }
    if (!aborted) flush(q_end);
    if (!SEG) break;
  }
  grid_launch_dependents();
  if (aborted) {
    if (warp == 0) block_drain(bars, S, k, issued, s, phase);
    if constexpr (CL) cluster_barrier();
    return;
  }
  if constexpr (ACC) {
    if constexpr (LN) {
      if (p.ws1) {
#pragma unroll
        for (int j = 0; j < NA1; ++j) io.partial(p.ws1 + grp * N + col0, j, acc1[j], false);
      }
    }
    if (p.ws2) {
#pragma unroll
      for (int j = 0; j < NA; ++j) io.partial(p.ws2 + grp * N + col0, j, acc2[j], false);
    }
  }
  if constexpr (CL) cluster_barrier();
}

// ---------------------------------------------------------------------------
// Launch shapes
// ---------------------------------------------------------------------------
// Launch a kernel given as the plain and the cluster instantiation (general
// form: the cluster one also for one CTA a row).  The smallest split of a row
// over 1, 2, 4 or 8 CTAs whose ring holds two stages; then as many CTAs per SM as
// registers (and, with weight gradients, the workspace's partial rows) allow, with
// the ring as deep as shared memory allows, up to about 128 KB of rows in flight
// per SM.
// `alts`: other shapes of the plain one, taken for a row in one CTA where its
// rows an SM at once, over the time each takes, are more: floor(warps / row's
// warps) / cost.  A thread's time goes as its columns and about 8 columns'
// worth of sums and barriers, times what the shape costs besides: one norm's
// backward reads and decodes twice (1.3), a forward in 96 registers is slower by
// a twentieth (1.05), with checkpoints it spills (1.2), and so does the general
// form (1.4).
template <class Fn>
struct BlockShape {
  Fn fn;
  BlockCta cta;
  double cost;
};
inline double block_rate(int64_t NL, const BlockCta& c, double cost) {
  const int64_t w = (NL + 32 * c.cols - 1) / (32 * c.cols);
  return w > c.warps || w * 32 > c.threads ? 0.0 : (double)(c.warps / w) / (cost * (c.cols + 8));
}
template <bool ALN, class Fn>
int launch_block(Fn plain, Fn split, BlockCta cta, std::initializer_list<BlockShape<Fn>> alts, BlockParams p, int es, bool qx, bool q8,
                 bool acc, const DevInfo& di, cudaStream_t st, int* grid) {
  const int vec = 16 / es;
  for (int ncl = 1; ncl <= 8; ncl *= 2) {
    if (di.tune_cluster > 0 && ncl != di.tune_cluster) continue;
    int64_t NL;   // columns of a slice (the general form's last one may have fewer)
    if (ALN) {
      if ((p.N / vec) % ncl) continue;
      NL = p.N / ncl;
      // a checkpoint's groups lie within a slice; where it is read (qx), a
      // slice's scales start and end on 16 bytes.  (Lengths that are not so split
      // take the general form: backward 4096 x 13824 342 us, 4096 x 16384 175.)
      if (ncl > 1 && q8 && NL % (qx ? 16 * kCkptGroup : kCkptGroup)) continue;
    } else {
      // slices of what a warp takes at 16 columns a lane (a checkpoint that is read
      // needs that); where the last would then be empty (8 of 24577 to 25088
      // columns), of 32 columns (always: 1024 x 40001 backward 344 -> 354 us)
      constexpr int64_t WARP = 16 * kCkptGroup;
      const int64_t each = (p.N + ncl - 1) / ncl;
      NL = ncl == 1 ? p.N : (each + WARP - 1) / WARP * WARP;
      if (!qx && NL * (ncl - 1) >= p.N) NL = (each + 31) / 32 * 32;
      if (NL * (ncl - 1) >= p.N) continue;
    }
    if (NL > kSliceCols) continue;
    Fn fn = !ALN || ncl > 1 ? split : plain;
    int cols = cta.cols;
    double best = block_rate(NL, cta, 1.0);
    for (const BlockShape<Fn>& alt : alts) {
      const double rate = ncl == 1 ? block_rate(NL, alt.cta, alt.cost) : 0.0;
      if (rate <= best) continue;
      best = rate;
      fn = alt.fn;
      cols = alt.cta.cols;
    }
    const int threads = (int)((NL + 32 * cols - 1) / (32 * cols)) * 32;
    p.part = (int)NL;
    // a stage, and the room (`off`) that the shape is chosen by
    uint32_t off = 0;
    p.stage_bytes = 0;
    for (int s = 0; s < kBlockStreams; ++s) {
      p.soff[s] = p.stage_bytes;
      if (!p.in[s] && !(s == SX && p.room_x)) continue;
      uint32_t len;
      if (qx && (s == SX || s == SH)) len = (uint32_t)((NL + 15) / 16 * 16 + (NL + 511) / 512 * 16);
      else len = ALN ? (uint32_t)(NL * es) : (uint32_t)((NL * es + 15) / 16 * 16 + 16);
      off += len;
      if (p.in[s]) p.stage_bytes += len;
    }
    const void* fp = reinterpret_cast<const void*>(fn);
    const KernelInfo ki = kernel_info(fp, di);
    if (ki.max_dyn < 0) return NORM_ERR_CUDA;
    const size_t least = kBlockHeader + 2 * (size_t)off;
    if (least > (size_t)ki.max_dyn) continue;
    const int nb = cached_occupancy(fp, di, threads, least);
    if (nb < 0) return NORM_ERR_CUDA;
    if (nb == 0) continue;
    int ctas = nb;
    if (di.tune_max_ctas > 0 && ctas > di.tune_max_ctas) ctas = di.tune_max_ctas;
    if (acc) {
      const int64_t per_sm = (di.max_partial_rows * ncl + di.sms - 1) / di.sms;
      if (per_sm >= 1 && ctas > per_sm) ctas = (int)per_sm;
    }
    // the deepest ring of stages of `bytes` that leaves room for n CTAs an SM: its
    // stages (0: not two) and shared memory
    size_t smem = 0;
    auto ring = [&](uint32_t bytes, int n) {
      const size_t two = kBlockHeader + 2 * (size_t)bytes;
      size_t room = (size_t)di.smem_per_sm / n;
      const size_t fixed_sm = (size_t)di.smem_reserved + 1536;   // reserved, and the static arrays
      room = room > fixed_sm ? room - fixed_sm : 0;
      if (room > (size_t)ki.max_dyn) room = (size_t)ki.max_dyn;
      if (n > 1 && room < two) return 0;
      if (room < two) room = two;
      int S = (int)((room - kBlockHeader) / bytes);
      const size_t inflight = (size_t)(di.tune_inflight_16k > 0 ? di.tune_inflight_16k : kInflightUnits) * 16384;
      const int cap = 1 + (int)(inflight / ((size_t)n * bytes));
      if (S > cap) S = cap > 2 ? cap : 2;
      if (S > kBlockMaxStages) S = kBlockMaxStages;
      if (di.tune_max_stages >= 2 && S > di.tune_max_stages) S = di.tune_max_stages;
      for (; S >= 2; --S) {
        smem = kBlockHeader + (size_t)S * bytes;
        const int fit = cached_occupancy(fp, di, threads, smem);
        if (fit < 0) return -1;
        if (fit >= n) return S;
      }
      return 0;
    };
    int S = 0;
    for (; ctas >= 1; --ctas) {
      S = ring(off, ctas);
      if (S < 0) return NORM_ERR_CUDA;
      if (S >= 2) break;
    }
    if (ctas < 1) continue;
    // row groups resident at once, held to the rows and the partial rows
    int64_t G = (int64_t)di.sms * ctas;
    if (ncl > 1) {
      G = cached_clusters(fp, di, threads, smem, ncl);
      if (G < 0) return NORM_ERR_CUDA;
      if (G == 0) continue;
    }
    // (room that no stream takes deepens the ring: 4096 x 4096 fp32 with a frozen
    // gate per token, three stages in place of two, 80 -> 69 us)
    if (p.stage_bytes < off) S = ring(p.stage_bytes, ctas);
    if (S < 2) return NORM_ERR_CUDA;
    if (G > p.M) G = p.M;
    if (acc && G > di.max_partial_rows) G = di.max_partial_rows;
    // a group counts its rows in 32 bits
    if ((p.M + G - 1) / G > (int64_t)INT32_MAX / 2) return NORM_ERR_TOO_LARGE;
    p.row_step = p.seg ? 1 : G;
    p.a_step = p.row_step * p.a_stride;
    p.b_step = p.row_step * p.b_stride;
    p.q_step = p.row_step * p.q_stride;
    p.dg_step = p.row_step * p.dg_stride;
    const int rc =
        launch_pdl_cluster(fn, dim3((unsigned)(G * ncl)), dim3((unsigned)threads), smem, ncl, st, p, S);
    if (rc == NORM_OK) *grid = (int)G;
    return rc;
  }
  return NORM_ERR_UNSUPPORTED_INTERNAL;
}

template <class T, int FORM, bool GROW, bool Q8>
int run_block_fwd(const BlockParams& p, const BlockFlags& f, const DevInfo& di, cudaStream_t st, int* grid) {
  constexpr int ES = (int)sizeof(T);
  using Fn = void (*)(const BlockParams, const int);
  int rc = NORM_ERR_UNSUPPORTED_INTERNAL;
  if (f.aligned && p.N % (16 / ES) == 0 && di.force_path != 2) {
    const BlockShape<Fn> narrow = {block_fwd_kernel<T, FORM, GROW, Q8, 2, true, false>, kNarrowCta, 1.0};
    BlockShape<Fn> alt = narrow;
    if constexpr (!one_norm(FORM))
      alt = {block_fwd_kernel<T, FORM, GROW, Q8, 1, true, false>, fwd_cta(FORM, Q8, 1, true),
             Q8 && FORM != kLn ? 1.2 : 1.05};
    rc = launch_block<true, Fn>(block_fwd_kernel<T, FORM, GROW, Q8, 0, true, false>,
                                block_fwd_kernel<T, FORM, GROW, Q8, 0, true, true>, fwd_cta(FORM, Q8, 0, true),
                                {alt, narrow}, p, ES, false, Q8, false, di, st, grid);
  }
  if (rc == NORM_ERR_UNSUPPORTED_INTERNAL) {
    constexpr int GF = FORM == kLn || FORM == kNorm ? FORM : kDynamic;
    Fn fn = block_fwd_kernel<T, GF, GROW, Q8, 0, false, true>;
    constexpr BlockCta cta = fwd_cta(GF, Q8, 0, false);
    if constexpr (Q8 && !one_norm(GF))
      rc = launch_block<false, Fn>(
          fn, fn, cta, {{block_fwd_kernel<T, GF, GROW, Q8, 1, false, true>, fwd_cta(GF, Q8, 1, false), 1.4}}, p, ES, false,
          Q8, false, di, st, grid);
    else
      rc = launch_block<false, Fn>(fn, fn, cta, {}, p, ES, false, Q8, false, di, st, grid);
  }
  return rc == NORM_ERR_UNSUPPORTED_INTERNAL ? NORM_ERR_TOO_LARGE : rc;
}

template <class T, int FORM, int GATE, bool Q8, bool ACC>
int run_block_bwd(const BlockParams& p, const BlockFlags& f, const DevInfo& di, cudaStream_t st, int* grid) {
  constexpr int ES = (int)sizeof(T);
  using Fn = void (*)(const BlockParams, const int);
  int rc = NORM_ERR_UNSUPPORTED_INTERNAL;
  if (f.aligned && p.N % (16 / ES) == 0 && di.force_path != 2) {
    const BlockShape<Fn> alt = {block_bwd_kernel<T, FORM, GATE, Q8, ACC, 1, true, false>, bwd_cta(FORM, 1, true),
                                one_norm(FORM) ? 1.3 : 1.0};
    BlockShape<Fn> narrow = alt;
    if constexpr (!ACC || (FORM != kLn && FORM != kNorm))
      narrow = {block_bwd_kernel<T, FORM, GATE, Q8, ACC, 2, true, false>, kNarrowCta, 1.0};
    rc = launch_block<true, Fn>(block_bwd_kernel<T, FORM, GATE, Q8, ACC, 0, true, false>,
                                block_bwd_kernel<T, FORM, GATE, Q8, ACC, 0, true, true>, bwd_cta(FORM, 0, true),
                                {alt, narrow}, p, ES, Q8, Q8, ACC, di, st, grid);
  }
  if (rc == NORM_ERR_UNSUPPORTED_INTERNAL) {
    constexpr int GF = FORM == kLn || FORM == kNorm ? FORM : kDynamic;
    Fn fn = block_bwd_kernel<T, GF, GATE, Q8, ACC, 0, false, true>;
    rc = launch_block<false, Fn>(
        fn, fn, bwd_cta(GF, 0, false),
        {{block_bwd_kernel<T, GF, GATE, Q8, ACC, 1, false, true>, bwd_cta(GF, 1, false), 1.4}}, p, ES, Q8, Q8, ACC, di, st,
        grid);
  }
  return rc == NORM_ERR_UNSUPPORTED_INTERNAL ? NORM_ERR_TOO_LARGE : rc;
}

}  // namespace gb300norm
