// Routing of tokens to experts: the choice and its weights, their gradient, and the order of the
// (token, choice) slots by expert.
#include "common.hpp"
#include "launch.hpp"
#include "pieces.hpp"

namespace nms {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kFltMax = 3.402823466e38f;

// Reductions over LPT consecutive lanes (16: one DPP row, 64: the wave); every lane gets the result.
template <int CTRL>
__device__ inline uint32_t dpp_row(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
template <int LPT, typename F>
__device__ inline float reduce_f32(float v, F f) {
  v = f(v, __uint_as_float(dpp_row<0x128>(__float_as_uint(v))));   // row_ror 8, 4, 2, 1
  v = f(v, __uint_as_float(dpp_row<0x124>(__float_as_uint(v))));
  v = f(v, __uint_as_float(dpp_row<0x122>(__float_as_uint(v))));
  v = f(v, __uint_as_float(dpp_row<0x121>(__float_as_uint(v))));
  if constexpr (LPT == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LPT>
__device__ inline float reduce_max(float v) {
  return reduce_f32<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
// Sums by rotation: the lanes add the same 16 terms in different orders, so lane 0's sum is taken.
template <int LPT>
__device__ inline float reduce_sum(float v, int lane) {
  v = reduce_f32<LPT>(v, [](float a, float b) { return a + b; });
  return __shfl(v, lane & ~(LPT - 1));
}
// A choice as one number: the order key in the high 32 of 62 bits, below it the complement of the
// expert's index, so that the largest is the best and on equal keys the lowest index.  Read as a double
// (positive and finite: the bits above are 0), so that one instruction takes the larger of two.
__device__ inline double choice(uint32_t key, int e) {
  const uint64_t b = ((uint64_t)key << 30) | (uint32_t)(1023 - e);
  return __builtin_bit_cast(double, key ? b : 0);
}
__device__ inline double larger(double a, double b) { return __builtin_fmax(a, b); }
template <int CTRL>
__device__ inline double larger_step(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 o = {dpp_row<CTRL>(b[0]), dpp_row<CTRL>(b[1])};
  return larger(v, __builtin_bit_cast(double, o));
}
template <int LPT>
__device__ inline double reduce_larger(double v) {
  v = larger_step<0x121>(larger_step<0x122>(larger_step<0x124>(larger_step<0x128>(v))));
  if constexpr (LPT == 64) {
    v = larger(v, __shfl_xor(v, 16));
    v = larger(v, __shfl_xor(v, 32));
  }
  return v;
}

// The two largest of two lanes' two largest.
template <int CTRL>
__device__ inline void merge_top2(float& t1, float& t2) {
  const float o1 = __uint_as_float(dpp_row<CTRL>(__float_as_uint(t1)));
  const float o2 = __uint_as_float(dpp_row<CTRL>(__float_as_uint(t2)));
  t2 = fmaxf(fmaxf(t2, o2), fminf(t1, o1));
  t1 = fmaxf(t1, o1);
}

// Unsigned key with the order of the floats (no NaN; +0 and -0 alike); every value but -infinity
// has a key above 0x007FFFFF, so 0 stands for "cannot be chosen".
__device__ inline uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A lane's EPL consecutive logits of one token; -infinity beyond E.  vec: the row and E allow whole
// vector loads.
template <typename T, int EPL>
__device__ inline void load_logits(const T* row, int e0, int E, bool vec, float (&v)[EPL]) {
  constexpr int PER = 16 / (int)sizeof(T) < EPL ? 16 / (int)sizeof(T) : EPL;   // elements a load
  if (vec) {
    if (e0 < E) {
#pragma unroll
      for (int i = 0; i < EPL; i += PER) {
        T b[PER];
        __builtin_memcpy(b, __builtin_assume_aligned(row + e0 + i, PER * sizeof(T)), sizeof(b));
#pragma unroll
        for (int q = 0; q < PER; ++q) v[i + q] = Elem<T>::to_f32(b[q]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = kNegInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = e0 + i < E ? Elem<T>::to_f32(row[e0 + i]) : kNegInf;
  }
  // NaN cannot be chosen, +infinity counts as the largest finite value
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = v[i] == v[i] ? fminf(v[i], kFltMax) : kNegInf;
}

// sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)): no overflow, and its first factor can be shifted.
__device__ inline float sigmoid_shifted(float l, float shift) {
  return expf(fminf(l, 0.f) - shift) / (1.f + expf(-fabsf(l)));
}

// LPT lanes per token, EPL consecutive experts per lane (LPT * EPL >= E), 64 / LPT tokens a wave.
// The k choices are k rounds of: each lane's best of its EPL keys, the best of the LPT lanes, its
// key cleared.  Slot j's id ends in lane j, which computes the weight.  What bounds it: a launch and
// one round trip to memory for few tokens (one of 64 experts, k 8: 3.0 us); for many, the rounds' vector
// instructions (8192 of 256 experts, k 8: 10.6 us).
template <typename T, int LPT, int EPL>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a, bool vec, bool vec_bias) {
  constexpr int TPW = 64 / LPT, ROW = LPT * EPL;
  __shared__ float lg[4 * TPW][ROW];
  __shared__ float cs[4 * TPW][ROW];
  __shared__ float gscore[4 * TPW][64];
  __shared__ uint8_t gkeep[4 * TPW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & (LPT - 1), slot_tok = wave * TPW + lane / LPT;
  const int64_t token = (int64_t)blockIdx.x * (4 * TPW) + slot_tok;
  const bool live = token < a.T;
  const T* row = (const T*)a.logits + (live ? token : a.T - 1) * a.ldl;
  const int e0 = li * EPL, E = a.E;

  float v[EPL];
  load_logits<T, EPL>(row, e0, E, vec, v);
#pragma unroll
  for (int i = 0; i < EPL; ++i) lg[slot_tok][e0 + i] = v[i];

  const bool grouped = a.groups > 1;
  float m = 0.f, Z = 1.f;
  if (!a.sigmoid && (a.bias || grouped || !a.renorm)) {
    float mx = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, v[i]);
    mx = reduce_max<LPT>(mx);
    m = mx > kNegInf ? mx : 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += expf(v[i] - m);
    z = reduce_sum<LPT>(z, lane);
    Z = z > 0.f ? z : 1.f;
  }

  uint32_t key[EPL];
  float c[EPL];
  if (a.bias || grouped) {
    float b[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = 0.f;
    if (vec_bias) {
      if (e0 < E) __builtin_memcpy(b, __builtin_assume_aligned(a.bias + e0, 16), sizeof(b));
    } else if (a.bias) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) b[i] = a.bias[e0 + i < E ? e0 + i : E - 1];
    }
    // reciprocals of one unit in the last place
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = __builtin_amdgcn_rcpf(1.f + expf(-v[i]));
    } else {
      const float inv = 1.f / Z;
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = expf(v[i] - m) * inv;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] += b[i];
      const bool ok = v[i] > kNegInf && c[i] > kNegInf;   // false for a NaN bias
      c[i] = ok ? c[i] : kNegInf;
      key[i] = ok ? order_key(a.bias ? c[i] : v[i]) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = v[i] > kNegInf ? order_key(v[i]) : 0u;
  }
  __syncthreads();

  if (grouped) {
    const int size = E / a.groups;
    // Registers where every group is a power of two of whole lanes and the groups fill the 16 lanes: E is
    // 64 or 256, and 2 to 16 groups.  8192 tokens of 256 experts in 8 groups 9.1 us, through LDS 11.0; 64
    // experts 5.2 and 5.8; 64 tokens of 256 6.8 and 9.0.  Other sizes take LDS (128 experts 10.6, 160 10.9).
    const int lanes = size / EPL;
    if (LPT == 16 && size == lanes * EPL && (lanes & (lanes - 1)) == 0 && lanes * a.groups == 16) {
      // in registers: a lane's two largest, merged over the group's lanes (xor 1, 2, then mirrors, which
      // reach the other half once the halves agree); then every lane sees the 15 others by rotation
      float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        t2 = fmaxf(t2, fminf(t1, c[i]));
        t1 = fmaxf(t1, c[i]);
      }
      if (lanes >= 2) merge_top2<0xB1>(t1, t2);
      if (lanes >= 4) merge_top2<0x4E>(t1, t2);
      if (lanes >= 8) merge_top2<0x141>(t1, t2);
      const float mine = a.group_top == 2 && t2 > kNegInf ? t1 + t2 : t1;
      const int g = li / lanes;
      float o = mine;
      int og = g, rank = 0;
      for (int r = 1; r < 16; ++r) {
        o = __uint_as_float(dpp_row<0x121>(__float_as_uint(o)));
        og = (int)dpp_row<0x121>((uint32_t)og);
        rank += (o > mine || (o == mine && og < g)) ? 1 : 0;   // each better group once per lane of it
      }
      if (rank >= a.topk_groups * lanes) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) cs[slot_tok][e0 + i] = c[i];
      __syncthreads();
      for (int g = li; g < a.groups; g += LPT) {
        float t1 = kNegInf, t2 = kNegInf;
        for (int j = 0, q = g % size; j < size; ++j, q = q + 1 == size ? 0 : q + 1) {   // staggered: LDS banks
          const float v1 = cs[slot_tok][g * size + q];
          t2 = fmaxf(t2, fminf(t1, v1));
          t1 = fmaxf(t1, v1);
        }
        gscore[slot_tok][g] = a.group_top == 2 && t2 > kNegInf ? t1 + t2 : t1;
      }
      __syncthreads();
      for (int g = li; g < a.groups; g += LPT) {
        const float mine = gscore[slot_tok][g];
        int rank = 0;
        for (int q = 0; q < a.groups; ++q) {
          const float o = gscore[slot_tok][q];
          rank += (o > mine || (o == mine && q < g)) ? 1 : 0;
        }
        gkeep[slot_tok][g] = rank < a.topk_groups;
      }
      __syncthreads();
      int g = e0 / size, left = size - e0 % size;   // this expert's group, and how many of it are left
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (e0 + i < E && !gkeep[slot_tok][g]) key[i] = 0u;
        if (--left == 0) {
          ++g;
          left = size;
        }
      }
    }
  }

  double pick[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) pick[i] = choice(key[i], e0 + i);
  int id = -1;
  for (int r = 0; r < a.k; ++r) {
    double best = pick[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = larger(best, pick[i]);
    best = reduce_larger<LPT>(best);
    const uint64_t b = __builtin_bit_cast(uint64_t, best);
    const int won = b ? 1023 - (int)(b & 1023) : -1;
    if (li == r) id = won;
    const int mine = won - e0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) pick[i] = mine == i ? 0.0 : pick[i];
  }

  const bool has = li < a.k && id >= 0;
  const float l = has ? lg[slot_tok][id] : kNegInf;
  float w;
  if (a.renorm) {
    // both scores divided by the same power of e, so that tiny scores keep their ratios
    const float peak = reduce_max<LPT>(has ? (a.sigmoid ? fminf(l, 0.f) : l) : kNegInf);
    const float r = has ? (a.sigmoid ? sigmoid_shifted(l, peak) : expf(l - peak)) : 0.f;
    const float sum = reduce_sum<LPT>(r, lane);
    w = has ? a.scale * (r / sum) : 0.f;
  } else {
    w = has ? a.scale * (a.sigmoid ? sigmoid_shifted(l, 0.f) : expf(l - m) / Z) : 0.f;
  }
  if (live && li < a.k) {
    a.ids[token * a.k + li] = id;
    a.weights[token * a.k + li] = w;
  }
}

// The same lanes and experts: the chosen entries are placed in an LDS row, and each lane adds the
// dense part (plain softmax only) to its experts and stores them.
template <typename T, int LPT, int EPL>
__global__ __launch_bounds__(256) void moe_route_bwd_kernel(const T* logits, int64_t ldl, int64_t Tn, int E, int sigmoid,
                                                            int k, int renorm, float scale, const int32_t* ids,
                                                            const float* weights, const float* dweights, T* dlogits,
                                                            int64_t lddl, bool vec_in, bool vec_out) {
  constexpr int TPW = 64 / LPT, ROW = LPT * EPL;
  __shared__ float buf[4 * TPW][ROW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & (LPT - 1), slot_tok = wave * TPW + lane / LPT;
  const int64_t tok = (int64_t)blockIdx.x * (4 * TPW) + slot_tok;
  const bool live = tok < Tn;
  const int64_t token = live ? tok : Tn - 1;
  const T* row = logits + token * ldl;
  const int e0 = li * EPL;

  int id = -1;
  float w = 0.f, dw = 0.f;
  if (li < k) {
    id = ids[token * k + li];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      w = weights[token * k + li];
      dw = dweights[token * k + li];
    }
  }
  const float wdw = w * dw;
  float g = 0.f, oneminus = 1.f, s[EPL];
  const bool dense = !sigmoid && !renorm;
  if (renorm || dense) g = reduce_sum<LPT>(wdw, lane);
  if (sigmoid && id >= 0) {
    float l = Elem<T>::to_f32(row[id]);
    oneminus = 1.f / (1.f + expf(l));
  }
  if (dense) {
    float v[EPL];
    load_logits<T, EPL>(row, e0, E, vec_in, v);
    float mx = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, v[i]);
    mx = reduce_max<LPT>(mx);
    const float m = mx > kNegInf ? mx : 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = expf(v[i] - m);
      z += s[i];
    }
    z = reduce_sum<LPT>(z, lane);
    const float gz = z > 0.f ? g / z : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= gz;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) buf[slot_tok][e0 + i] = 0.f;
  __syncthreads();
  if (id >= 0) buf[slot_tok][id] = (renorm ? w * (dw - g / scale) : wdw) * oneminus;
  __syncthreads();
  if (!live) return;
  T* out = dlogits + token * lddl;
  T o[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float d = buf[slot_tok][e0 + i] - (dense ? s[i] : 0.f);
    if constexpr (sizeof(T) == 2) o[i] = f32_to_bf16_rne(d); else o[i] = __float_as_uint(d);
  }
  if (vec_out) {
    constexpr int PER = 16 / (int)sizeof(T) < EPL ? 16 / (int)sizeof(T) : EPL;
    if (e0 < E) {
#pragma unroll
      for (int i = 0; i < EPL; i += PER)
        __builtin_memcpy(__builtin_assume_aligned(out + e0 + i, PER * sizeof(T)), o + i, PER * sizeof(T));
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i < E) out[e0 + i] = o[i];
  }
}

bool rows_vec(const void* p, int64_t ld, int es, int E, int epl) {
  return E % epl == 0 && (ld * es) % 16 == 0 && (uintptr_t)p % 16 == 0;
}

template <typename T, int LPT, int EPL>
hipError_t run_route(const RouteArgs& a, hipStream_t s) {
  const int per = 4 * (64 / LPT);
  hipLaunchKernelGGL((moe_route_kernel<T, LPT, EPL>), dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, s, a,
                     rows_vec(a.logits, a.ldl, sizeof(T), a.E, EPL),
                     a.bias && a.E % EPL == 0 && (uintptr_t)a.bias % 16 == 0);
  return hipGetLastError();
}

template <typename T>
hipError_t route_piece(const RouteArgs& a, hipStream_t s) {
  if (a.k <= 16 && a.E <= 64) return run_route<T, 16, 4>(a, s);
  if (a.k <= 16 && a.E <= 256) return run_route<T, 16, 16>(a, s);
  if (a.E <= 256) return run_route<T, 64, 4>(a, s);
  return run_route<T, 64, 16>(a, s);
}

template <typename T>
hipError_t route_t(const RouteArgs& a, hipStream_t s) {
  return in_pieces(a.T, kPieceRows, [&](int64_t t0, int64_t n) {
    RouteArgs p = a;
    p.logits = (const T*)a.logits + t0 * a.ldl;
    p.T = n;
    p.ids += t0 * a.k;
    p.weights += t0 * a.k;
    return route_piece<T>(p, s);
  });
}

template <typename T, int LPT, int EPL>
hipError_t run_bwd(const T* logits, int64_t ldl, int64_t Tn, int E, int sigmoid, int k, int renorm, float scale,
                   const int32_t* ids, const float* w, const float* dw, T* dl, int64_t lddl, hipStream_t s) {
  const int per = 4 * (64 / LPT);
  hipLaunchKernelGGL((moe_route_bwd_kernel<T, LPT, EPL>), dim3((unsigned)((Tn + per - 1) / per)), dim3(256), 0, s,
                     logits, ldl, Tn, E, sigmoid, k, renorm, scale, ids, w, dw, dl, lddl,
                     rows_vec(logits, ldl, sizeof(T), E, EPL), rows_vec(dl, lddl, sizeof(T), E, EPL));
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_piece(const T* logits, int64_t ldl, int64_t Tn, int E, int sigmoid, int k, int renorm, float scale,
                 const int32_t* ids, const float* w, const float* dw, T* dl, int64_t lddl, hipStream_t s) {
  if (k <= 16 && E <= 64) return run_bwd<T, 16, 4>(logits, ldl, Tn, E, sigmoid, k, renorm, scale, ids, w, dw, dl, lddl, s);
  if (k <= 16 && E <= 256)
    return run_bwd<T, 16, 16>(logits, ldl, Tn, E, sigmoid, k, renorm, scale, ids, w, dw, dl, lddl, s);
  if (E <= 256) return run_bwd<T, 64, 4>(logits, ldl, Tn, E, sigmoid, k, renorm, scale, ids, w, dw, dl, lddl, s);
  return run_bwd<T, 64, 16>(logits, ldl, Tn, E, sigmoid, k, renorm, scale, ids, w, dw, dl, lddl, s);
}

template <typename T>
hipError_t bwd_t(const T* logits, int64_t ldl, int64_t Tn, int E, int sigmoid, int k, int renorm, float scale,
                 const int32_t* ids, const float* w, const float* dw, T* dl, int64_t lddl, hipStream_t s) {
  return in_pieces(Tn, kPieceRows, [&](int64_t t0, int64_t n) {
    return bwd_piece<T>(logits + t0 * ldl, ldl, n, E, sigmoid, k, renorm, scale, ids + t0 * k, w + t0 * k, dw + t0 * k,
                        dl + t0 * lddl, lddl, s);
  });
}

// ---------------------------------------------------------------------------
// moe_plan: a stable counting sort of the slots by expert.  The slots are cut into chunks (one
// workgroup each); with more than one chunk a first kernel counts every chunk's slots per expert,
// and each workgroup of the second adds up the counts before its own.  Inside a chunk each wave
// takes a contiguous part, 64 slots at a time: lanes of equal expert find each other by ballots over
// the bits of the id, and a lane's place is the wave's counter for the expert plus the number of
// such lanes below it.  Integer counts only: the result does not depend on the order of threads.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int64_t kPlanChunk = 4096;   // of a single workgroup
constexpr int64_t kPlanSmall = 2048;   // of one of many

int64_t plan_chunk(int64_t n) {
  // at most 256 chunks: a workgroup of the second kernel reads every chunk's counts
  if (n <= kPlanChunk) return kPlanChunk;
  const int64_t c = (n + 255) / 256;
  return c <= kPlanSmall ? kPlanSmall : (c + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

__global__ __launch_bounds__(kPlanThreads) void moe_plan_count_kernel(const int32_t* ids, int64_t n, int E,
                                                                      int64_t chunk, int32_t* work) {
  extern __shared__ int32_t cnt[];
  for (int e = threadIdx.x; e < E; e += kPlanThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) work[(int64_t)blockIdx.x * E + e] = cnt[e];
}

__global__ __launch_bounds__(kPlanThreads) void moe_plan_place_kernel(const int32_t* ids, int64_t n, int E, int bits,
                                                                      int align, int64_t chunk, int nchunks,
                                                                      int32_t* offsets, int32_t* counts, int32_t* src,
                                                                      int64_t rows, int32_t* pos, const int32_t* work) {
  extern __shared__ int32_t smem[];
  int32_t* hist = smem;                       // [waves][E]: a wave's counts, then its next rows
  int32_t* scan = hist + kPlanWaves * E;      // [1024] padded counts, summed up to and including e
  int32_t* lows = scan + kPlanThreads;        // [1024]
  int32_t* total = lows + kPlanThreads;       // [E]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  const int64_t part = chunk / kPlanWaves;    // a multiple of 64
  const int64_t wlo = lo + wave * part, whi = wlo + part < hi ? wlo + part : hi;

  for (int i = tid; i < kPlanWaves * E; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 64) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&hist[wave * E + e], 1);
  }
  __syncthreads();
  int before = 0, mine = 0;
  int own[kPlanWaves];   // the waves' counts of expert tid
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) own[w] = hist[w * E + tid];
    if (nchunks == 1) {
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) mine += own[w];
    }
  }
  if (nchunks > 1) {
    // the counts of all chunks and of those before this one: E experts x as many parts as threads allow,
    // eight loads in flight each, added up through LDS (scan and the space behind it)
    const int parts = kPlanThreads / E < 16 ? kPlanThreads / E : 16;   // E <= 1024
    const int e = tid % E, part = tid / E;
    int sum = 0, low = 0;
    if (part < parts) {
      for (int c0 = part; c0 < nchunks; c0 += 8 * parts) {
        int v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = c0 + u * parts < nchunks ? work[(int64_t)(c0 + u * parts) * E + e] : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          sum += v[u];
          low += c0 + u * parts < (int)blockIdx.x ? v[u] : 0;
        }
      }
    }
    scan[tid] = sum;
    lows[tid] = low;
    __syncthreads();
    if (tid < E)
      for (int q = 0; q < parts; ++q) {
        mine += scan[q * E + tid];
        before += lows[q * E + tid];
      }
    __syncthreads();
  }
  if (tid < E) total[tid] = mine;
  const int padded = (mine + align - 1) & ~(align - 1);
  // inclusive sum of the padded counts over the experts: within waves, then over the waves
  int inc = padded;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  scan[tid] = inc;
  __syncthreads();
  int carry = lane < wave ? scan[lane * 64 + 63] : 0;
#pragma unroll
  for (int d = 8; d > 0; d /= 2) carry += __shfl_xor(carry, d);
  carry = __shfl(carry, 0);
  __syncthreads();
  inc += carry;
  scan[tid] = inc;
  if (tid < E) {
    int base = inc - padded + before;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      hist[w * E + tid] = base;
      base += own[w];
    }
    if (blockIdx.x == 0) {
      offsets[tid + 1] = inc;
      counts[tid] = mine;
      if (tid == 0) offsets[0] = 0;
    }
  }
  __syncthreads();
  volatile int32_t* next = hist + wave * E;
  for (int64_t i = wlo; i < whi; i += 64) {
    const int64_t slot = i + lane;
    const bool in = slot < whi;
    int e = in ? ids[slot] : -1;
    const bool ok = e >= 0 && e < E;
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t one = __ballot(ok && ((e >> b) & 1));
      same &= ((e >> b) & 1) ? one : ~one;
    }
    int p = -1;
    if (ok) {
      const int below = __popcll(same & ((uint64_t(1) << lane) - 1));
      p = next[e] + below;                                                 // all lanes read ...
      __builtin_amdgcn_wave_barrier();
      if (below == 0) next[e] = p + __popcll(same);                        // ... before the first of each expert moves on
      src[p] = (int32_t)slot;
    }
    __builtin_amdgcn_wave_barrier();
    if (in) pos[slot] = p;
  }
  // padding rows of the experts, and the rows behind the last expert
  for (int e = (int)blockIdx.x * kPlanWaves + wave; e < E; e += nchunks * kPlanWaves) {
    const int end = scan[e];
    const int first = (e ? scan[e - 1] : 0) + total[e];
    for (int r = first + lane; r < end; r += 64) src[r] = -1;
  }
  for (int64_t r = scan[E - 1] + (int64_t)blockIdx.x * kPlanThreads + tid; r < rows; r += (int64_t)nchunks * kPlanThreads)
    src[r] = -1;
}

}  // namespace

hipError_t launch_moe_route(int dt, const RouteArgs& a, hipStream_t s) {
  return dt == DT_BF16 ? route_t<uint16_t>(a, s) : route_t<uint32_t>(a, s);
}

hipError_t launch_moe_route_bwd(int dt, const void* logits, int64_t ldl, int64_t T, int E, int sigmoid, int k, int renorm,
                                float scale, const int32_t* ids, const float* weights, const float* dweights,
                                void* dlogits, int64_t lddl, hipStream_t s) {
  if (dt == DT_BF16)
    return bwd_t<uint16_t>((const uint16_t*)logits, ldl, T, E, sigmoid, k, renorm, scale, ids, weights, dweights,
                           (uint16_t*)dlogits, lddl, s);
  return bwd_t<uint32_t>((const uint32_t*)logits, ldl, T, E, sigmoid, k, renorm, scale, ids, weights, dweights,
                         (uint32_t*)dlogits, lddl, s);
}

int64_t moe_plan_work_bytes(int64_t n, int64_t E) {
  const int64_t chunk = plan_chunk(n), nchunks = (n + chunk - 1) / chunk;
  return nchunks > 1 ? nchunks * E * 4 : 0;
}

hipError_t launch_moe_plan(const int32_t* ids, int64_t n, int E, int align, int32_t* offsets, int32_t* counts,
                           int32_t* src, int64_t rows, int32_t* pos, int32_t* work, hipStream_t s) {
  const int64_t chunk = plan_chunk(n);
  const int nchunks = (int)((n + chunk - 1) / chunk);
  if (nchunks > 1)
    hipLaunchKernelGGL(moe_plan_count_kernel, dim3(nchunks), dim3(kPlanThreads), E * 4, s, ids, n, E, chunk, work);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  const size_t lds = ((size_t)kPlanWaves * E + 2 * kPlanThreads + E) * 4;
  (void)hipFuncSetAttribute((const void*)moe_plan_place_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  hipLaunchKernelGGL(moe_plan_place_kernel, dim3(nchunks), dim3(kPlanThreads), lds, s, ids, n, E, bits,
                     align, chunk, nchunks, offsets, counts, src, rows, pos, work);
  return hipGetLastError();
}

}  // namespace nms
