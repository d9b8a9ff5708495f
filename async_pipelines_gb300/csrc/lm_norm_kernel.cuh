// Dropout, and the root-mean-square norm with the residual's addition,
// forward and backward: kernels that read each value once and are bound by
// memory.
//
//   dropout        d(x) = keep * x / (1 - p)
//   forward        h = residual + d(x);  r = 1 / sqrt(mean(h^2) + eps);
//                  y = h * r * weight  (in the type of x, or in e4m3 with a
//                  scale for each row or each 128 columns)
//   backward       a = dy * weight;  n = h * r;
//                  dres = dh + r * (a - n * mean(a * n));
//                  dx = keep * dres / (1 - p);  dweight = sum over rows dy * n
//
// A row belongs to a team of threads that hold it in registers, 8 columns (a
// "group", 16 bytes of a 16-bit type) at a time: group k * team + t is thread
// t's k-th, so that a warp's accesses are contiguous. The row's statistics
// are reduced over the team in 32 bits and the row is never read again.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx.cuh"
#include "watchdog.cuh"

namespace gws {

constexpr int GROUP = 8;                 // columns of a group; Philox words of a counter
constexpr int QUANT_GROUP = 128;         // columns of one scale (Q == 2)
constexpr int MAX_VPT = 4;               // groups a thread holds
constexpr float E4M3_MAX = 448.0f;       // largest finite e4m3

// ------------------------------------------------------------ generator

// Philox4x32 with ten rounds (J. Salmon et al., "Parallel random numbers: as
// easy as 1, 2, 3", 2011): the key is the seed, the counter's low 64 bits are
// given and its high ones 0. The 128 bits serve the 8 columns of a group, 16
// bits each, lowest first: half the rounds' cost of 32 bits a column (which
// would take more issue slots than dropout's 4 bytes of traffic a column
// leave), for a p that is a multiple of 2^-16.
//
// N counters at a time: they share the rounds' keys, and the rounds of one fill
// the latency of the others'.
template <int N>
__device__ __forceinline__ void philox(const uint64_t (&counter)[N], uint64_t seed,
                                       uint32_t (&words)[N][4]) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    words[n][0] = static_cast<uint32_t>(counter[n]);
    words[n][1] = static_cast<uint32_t>(counter[n] >> 32);
    words[n][2] = words[n][3] = 0;
  }
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t(&c)[4] = words[n];
      const uint64_t m0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
      const uint64_t m1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
      c[0] = static_cast<uint32_t>(m1 >> 32) ^ c[1] ^ k0;
      c[1] = static_cast<uint32_t>(m1);
      c[2] = static_cast<uint32_t>(m0 >> 32) ^ c[3] ^ k1;
      c[3] = static_cast<uint32_t>(m0);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// What a launch's dropout is: a column is kept, and scaled, where its word,
// shifted to the top of 32 bits, is above `limit`.
struct Dropout {
  const uint64_t* rng;   // device: seed, first counter (readable, if unused, without dropout)
  int on;
  uint32_t limit;        // (round(65536 p) << 16) - 1
  float scale;           // 65536 / (65536 - round(65536 p)); 0 where all is dropped
};

// v = d(v) for N groups by their words. A dropped value is 0 whatever it was.
// Words are compared in the upper half of a register: the high one as it
// stands (what is below it cannot change the verdict), the low one shifted up.
template <int N>
__device__ __forceinline__ void drop_by(const Dropout& d, const uint32_t (&words)[N][4],
                                        float (&v)[N][GROUP]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[n][2 * i] = (words[n][i] << 16) > d.limit ? v[n][2 * i] * d.scale : 0.0f;
      v[n][2 * i + 1] = words[n][i] > d.limit ? v[n][2 * i + 1] * d.scale : 0.0f;
    }
}

// v = d(v) for N groups at their counters.
template <int N>
__device__ __forceinline__ void drop_groups(const Dropout& d, uint64_t seed,
                                            const uint64_t (&counter)[N], float (&v)[N][GROUP]) {
  uint32_t words[N][4];
  philox(counter, seed, words);
  drop_by(d, words, v);
}

// ------------------------------------------------------------ groups

// A group as it lies in memory, and its values in 32 bits.
template <typename T>
struct alignas(16) Raw {
  uint4 w[sizeof(T) * GROUP / 16];
};

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& raw, float (&v)[GROUP]) {
  const uint32_t w[4] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<__half>& raw, float (&v)[GROUP]) {
  const uint32_t w[4] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const Raw<float>& raw, float (&v)[GROUP]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(raw.w[i].x);
    v[4 * i + 1] = __uint_as_float(raw.w[i].y);
    v[4 * i + 2] = __uint_as_float(raw.w[i].z);
    v[4 * i + 3] = __uint_as_float(raw.w[i].w);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The group's values rounded to T.
template <typename T>
__device__ __forceinline__ Raw<T> pack(const float (&v)[GROUP]) {
  Raw<T> raw;
  if constexpr (sizeof(T) == 2) {
    raw.w[0] = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                          pack2(v[6], v[7], T()));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      raw.w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                            __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  }
  return raw;
}

__device__ __forceinline__ float round_to(float v, float) { return v; }
__device__ __forceinline__ __nv_bfloat16 round_to(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }
__device__ __forceinline__ __half round_to(float v, __half) { return __float2half_rn(v); }

// Element i of a group in registers: its bits, and a group made of them. (By
// shifts, so that the group stays in registers.)
template <typename T>
__device__ __forceinline__ uint32_t bits_of(const Raw<T>& raw, int i) {
  const uint32_t w[8] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w,
                         raw.w[sizeof(T) / 4].x, raw.w[sizeof(T) / 4].y,
                         raw.w[sizeof(T) / 4].z, raw.w[sizeof(T) / 4].w};
  return sizeof(T) == 4 ? w[i] : (w[i / 2] >> (16 * (i % 2))) & 0xFFFFu;
}
template <typename T>
__device__ __forceinline__ Raw<T> from_bits(const uint32_t (&e)[GROUP]) {
  Raw<T> raw;
  if constexpr (sizeof(T) == 2) {
    raw.w[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  } else {
    raw.w[0] = make_uint4(e[0], e[1], e[2], e[3]);
    raw.w[1] = make_uint4(e[4], e[5], e[6], e[7]);
  }
  return raw;
}

template <int N>
struct Int {
  static constexpr int value = N;
};

template <int SIZE>
struct Bits;
template <>
struct Bits<2> { using type = uint16_t; };
template <>
struct Bits<4> { using type = uint32_t; };

// Two fp32 values in a register pair, for the instructions that take two at
// once: the gradient's arithmetic would else need as many issue slots as its
// memory traffic leaves.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 values_of(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& raw, Pair (&v)[GROUP / 2]) {
  float f[GROUP];
  unpack(raw, f);
#pragma unroll
  for (int i = 0; i < GROUP / 2; ++i) v[i] = pair_of(f[2 * i], f[2 * i + 1]);
}

// How a kernel's rows lie, and whether values are dropped. FAST: every row of
// every matrix starts on a 16-byte boundary and ends with a whole group. DROP
// is FAST with dropout: the generator's rounds only overlap the loads around
// them where no branch stands before them (8192 x 8192 bf16, dropout alone: 55
// us behind a branch, 42 without; the copy alone takes 40). ANY is the rest, with
// dropout behind a branch.
enum Path { ANY = 0, FAST = 1, DROP = 2 };

// out = the bytes [by, by + 4 W) of `in`, 0 < by < 16. A warp's groups are mostly
// of one row, so that `by` is one and the branches are taken together.
template <int W>
__device__ __forceinline__ void shift_bytes(const uint32_t (&in)[W + 4], int by, uint32_t (&out)[W]) {
  const int bits = (by & 3) * 8;
  auto from = [&](auto first) {
    constexpr int F = decltype(first)::value;
#pragma unroll
    for (int i = 0; i < W; ++i)
      out[i] = __funnelshift_r(in[i + F], in[i + F + 1 < W + 4 ? i + F + 1 : W + 3], bits);
  };
  switch (by >> 2) {
    case 0: from(Int<0>()); break;
    case 1: from(Int<1>()); break;
    case 2: from(Int<2>()); break;
    default: from(Int<3>()); break;
  }
}

template <typename T>
constexpr int WORDS = sizeof(T) * GROUP / 4;   // of a group

template <typename T>
__device__ __forceinline__ void words_of(const Raw<T>& raw, uint32_t (&w)[WORDS<T>]) {
#pragma unroll
  for (int i = 0; i < WORDS<T> / 4; ++i) {
    w[4 * i] = raw.w[i].x;
    w[4 * i + 1] = raw.w[i].y;
    w[4 * i + 2] = raw.w[i].z;
    w[4 * i + 3] = raw.w[i].w;
  }
}

// A row of a matrix, and whether the matrix has at least 16 bytes before and
// after it (which may then be read along with it).
template <typename T>
struct Row {
  const T* at;
  bool before, after;
};
template <typename T>
__device__ __forceinline__ Row<T> row_of(const void* first, int64_t row, int64_t rows, int64_t ld) {
  const bool far = ld * sizeof(T) >= 16;
  return {static_cast<const T*>(first) + row * ld, far && row > 0, far && row + 1 < rows};
}

// The column at which group `g` of a row begins (the row's end for a thread without a
// group), and whether `n` columns from c on are all in the row. Rows have up to 2^31 - 1
// columns, so neither a group past the last nor c + n may be formed in 32 bits: they wrap,
// and a thread without a group would store below the row.
__host__ __device__ constexpr int column_of(int g, int groups, int cols) {
  return g < groups ? g * GROUP : cols;
}
__host__ __device__ constexpr bool has_columns(int c, int n, int cols) { return cols - c >= n; }

// Columns [c, c + 8) of a row whose end is `cols`; past it zeros. WHOLE (not
// ANY): a group moves in 16-byte pieces and nothing is tested. Else a group that
// does not start on a 16-byte boundary is cut out of the 16-byte pieces around it,
// where those lie within the matrix; at its two ends and the row's, single
// elements (which took twice the time for all of 8192 x 8191 bf16).
template <bool WHOLE, typename T>
__device__ __forceinline__ Raw<T> load_group(const Row<T>& row, int c, int cols) {
  const auto* src = reinterpret_cast<const typename Bits<sizeof(T)>::type*>(row.at) + c;
  constexpr int PIECES = WORDS<T> / 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(src);
  const int off = static_cast<int>(at & 15);
  const bool whole = has_columns(c, GROUP, cols);
  Raw<T> raw;
  if (WHOLE || (whole && off == 0)) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) raw.w[i] = reinterpret_cast<const uint4*>(src)[i];
  } else if (whole && (c > 0 || row.before) &&
             (has_columns(c, 2 * GROUP, cols) || row.after)) {
    uint32_t in[WORDS<T> + 4], out[WORDS<T>];
#pragma unroll
    for (int i = 0; i <= PIECES; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(at - off)[i];
      in[4 * i] = v.x;
      in[4 * i + 1] = v.y;
      in[4 * i + 2] = v.z;
      in[4 * i + 3] = v.w;
    }
    shift_bytes<WORDS<T>>(in, off, out);
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      raw.w[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
  } else {
    uint32_t e[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) e[i] = c + i < cols ? src[i] : 0u;
    raw = from_bits<T>(e);
  }
  return raw;
}

// Fetches the group into the cache, without waiting: the general path's loads
// take their data apart one after the other, so what they find there counts.
template <typename T>
__device__ __forceinline__ void prefetch_group(const Row<T>& row, int c) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(row.at + c));
}

// The bytes [from, 4 W) of w, to an address `to` that they bring to a 16-byte
// boundary: in pieces that grow with its alignment.
template <int W>
__device__ __forceinline__ void store_lead(uintptr_t to, const uint32_t (&w)[W]) {
  auto word = [&](int byte) { return __funnelshift_r(w[byte >> 2 & 3], w[((byte >> 2) + 1) & 3], (byte & 3) * 8); };
  int at = 0;
  if (to & 1) {
    *reinterpret_cast<uint8_t*>(to) = static_cast<uint8_t>(w[0]);
    at = 1;
  }
  if ((to + at) & 2) {
    *reinterpret_cast<uint16_t*>(to + at) = static_cast<uint16_t>(word(at));
    at += 2;
  }
  if ((to + at) & 4) {
    *reinterpret_cast<uint32_t*>(to + at) = word(at);
    at += 4;
  }
  if constexpr (W > 2)
    if ((to + at) & 8) *reinterpret_cast<uint2*>(to + at) = make_uint2(word(at), word(at + 4));
}

// The first `n` bytes of w to a 16-byte (W == 2: 8-byte) boundary.
template <int W>
__device__ __forceinline__ void store_tail(uintptr_t to, const uint32_t (&w)[W], int n) {
  int at = 0;
  if constexpr (W > 2)
    if (n & 8) {
      *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      at = 8;
    }
  if (n & 4) {
    *reinterpret_cast<uint32_t*>(to + at) = w[(at >> 2) & (W - 1)];
    at += 4;
  }
  const uint32_t last = w[(at >> 2) & (W - 1)];
  if (n & 2) {
    *reinterpret_cast<uint16_t*>(to + at) = static_cast<uint16_t>(last);
    at += 2;
  }
  if (n & 1) *reinterpret_cast<uint8_t*>(to + at) = static_cast<uint8_t>(last >> (n & 2 ? 16 : 0));
}

// Stores columns [c, c + 8) (as many as there are) of thread t's group of a row of
// `team` threads; WHOLE needs no other thread. Else the whole warp has to call it,
// threads without a group with c >= cols: neighbouring threads hold neighbouring
// groups, and where these do not start on a 16-byte boundary each thread stores the
// 16-byte pieces that end in its group, with the rest of its left neighbour's; the
// bytes at a warp's two ends go in smaller pieces, and a row's last group element by
// element.
template <bool WHOLE, typename T>
__device__ __forceinline__ void store_group(T* row, int c, int cols, int t, int team,
                                            const Raw<T>& raw) {
  auto* dst = reinterpret_cast<typename Bits<sizeof(T)>::type*>(row) + c;
  constexpr int PIECES = WORDS<T> / 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(dst);
  const int off = static_cast<int>(at & 15);   // the same for all groups of the row
  if constexpr (WHOLE) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) reinterpret_cast<uint4*>(dst)[i] = raw.w[i];
  } else {
    uint32_t own[WORDS<T>], in[WORDS<T> + 4], out[WORDS<T>];
    words_of(raw, own);
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = __shfl_up_sync(0xffffffffu, own[WORDS<T> - 4 + i], 1);
    const bool whole = has_columns(c, GROUP, cols);
    if (off == 0 && whole) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) reinterpret_cast<uint4*>(dst)[i] = raw.w[i];
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool left = lane > 0 && t > 0, right = lane < 31 && t + 1 < team;
    const int lead = (16 - off) / static_cast<int>(sizeof(T));   // elements up to the boundary
    if (off != 0 && whole) {
#pragma unroll
      for (int i = 0; i < WORDS<T>; ++i) in[4 + i] = own[i];
      shift_bytes<WORDS<T>>(in, 16 - off, out);
#pragma unroll
      for (int k = 0; k < PIECES; ++k)
        if (k > 0 || left)
          reinterpret_cast<uint4*>(at - off)[k] =
              make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]);
      if (!left) {
        const uint32_t first[4] = {own[0], own[1], own[2], own[3]};
        store_lead<4>(at, first);
      }
      // The right neighbour stores the piece that begins here, if all of it is there.
      if (!(right && has_columns(c, GROUP + lead, cols))) {
        uint32_t end[8], rest[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          end[i] = own[WORDS<T> - 4 + i];
          end[4 + i] = 0;
        }
        shift_bytes<4>(end, 16 - off, rest);
        store_tail<4>(at - off + 16 * PIECES, rest, off);
      }
      return;
    }
    if (c >= cols) return;
    // The row's last group, not whole: what the left neighbour begins, if all of
    // that piece is there, and the rest by elements.
    int from = 0;
    if (off != 0 && left && has_columns(c, lead, cols)) {
#pragma unroll
      for (int i = 0; i < WORDS<T>; ++i) in[4 + i] = own[i];
      shift_bytes<WORDS<T>>(in, 16 - off, out);
      *reinterpret_cast<uint4*>(at - off) = make_uint4(out[0], out[1], out[2], out[3]);
      from = lead;
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
      if (i >= from && c + i < cols)
        dst[i] = static_cast<typename Bits<sizeof(T)>::type>(bits_of(raw, i));
  }
}

// The same for the 8 bytes of an e4m3 group and pieces of 8 bytes.
template <bool WHOLE>
__device__ __forceinline__ void store_bytes(uint8_t* row, int c, int cols, int t, int team,
                                            uint2 raw) {
  uint8_t* dst = row + c;
  const uintptr_t at = reinterpret_cast<uintptr_t>(dst);
  const int off = static_cast<int>(at & 7), lead = 8 - off;
  if constexpr (WHOLE) {
    *reinterpret_cast<uint2*>(dst) = raw;
  } else {
    using Word = unsigned long long;
    const Word own = raw.x | static_cast<Word>(raw.y) << 32;
    const Word other = __shfl_up_sync(0xffffffffu, own, 1);
    const bool whole = has_columns(c, GROUP, cols);
    if (off == 0 && whole) {
      *reinterpret_cast<uint2*>(dst) = raw;
      return;
    }
    if (c >= cols) return;
    const int lane = threadIdx.x & 31;
    const bool left = off != 0 && lane > 0 && t > 0 && has_columns(c, lead, cols);
    if (left) *reinterpret_cast<Word*>(at - off) = own << (8 * off) | other >> (8 * lead);
    if (off != 0 && whole) {
      if (!left) {
        const uint32_t first[4] = {raw.x, raw.y, 0, 0};
        int n = 0;   // up to the 8-byte boundary
        if (at & 1) {
          dst[0] = static_cast<uint8_t>(raw.x);
          n = 1;
        }
        if ((at + n) & 2) {
          *reinterpret_cast<uint16_t*>(dst + n) = static_cast<uint16_t>(raw.x >> (8 * n));
          n += 2;
        }
        if ((at + n) & 4)
          *reinterpret_cast<uint32_t*>(dst + n) = __funnelshift_r(first[0], first[1], 8 * n);
      }
      if (!(lane < 31 && t + 1 < team && has_columns(c, GROUP + lead, cols))) {
        const Word end = own >> (8 * lead);
        const uint32_t rest[2] = {static_cast<uint32_t>(end), static_cast<uint32_t>(end >> 32)};
        store_tail<2>(at + lead, rest, off);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
      if (i >= (left ? lead : 0) && c + i < cols)
        dst[i] = static_cast<uint8_t>((i < 4 ? raw.x : raw.y) >> (8 * (i % 4)));
  }
}

// The e4m3 roundings of v / scale, lowest column first. A product with 1 / scale is off by
// a unit of the last place or two, which moves a quotient that lies between two e4m3 values
// (25 of scale 7 to 26, not 24). So the quotients are put between products with a smaller and
// a larger factor than 1 / scale: where the two round alike, so does what lies between
// them, and only else (one group in 10^5) are there divisions. (8192 x 8192 bf16, a scale a
// row: 75 us, 90 with divisions throughout, 70 with the product that rounds some wrongly.)
__device__ __forceinline__ uint2 quotients(const float (&v)[GROUP], float scale) {
  auto e4m3 = [](const float (&q)[GROUP]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
  };
  // 1 / scale and each factor are off by at most 2^-24 of themselves
  const float inv = 1.0f / scale;
  auto times = [&](float factor) {
    const Pair f = pair_of(factor, factor);
    float q[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; i += 2) {
      const float2 two = values_of(mul2(pair_of(v[i], v[i + 1]), f));
      q[i] = two.x;
      q[i + 1] = two.y;
    }
    return e4m3(q);
  };
  const uint2 least = times(inv * (1.0f - 0x1p-22f)), most = times(inv * (1.0f + 0x1p-22f));
  if (least.x == most.x && least.y == most.y) return least;
  float q[GROUP];
#pragma unroll
  for (int i = 0; i < GROUP; ++i) q[i] = v[i] / scale;
  return e4m3(q);
}

// ------------------------------------------------------------ reductions

// The larger, or NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct SumMax {
  float sum, max;
};

// The sum (and the largest) over a team: a warp, or a whole block of `warps`
// warps through `box` (one slot a warp; a block's next use of the same box
// needs a barrier in between). Each thread adds the warps' sums in the same
// order, so the result does not depend on timing.
template <bool MAX>
__device__ __forceinline__ SumMax reduce_team(SumMax v, int warps, SumMax* box) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    if (MAX) v.max = max_nan(v.max, __shfl_xor_sync(0xffffffffu, v.max, o));
  }
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
  __syncthreads();
  SumMax all = box[0];
  for (int w = 1; w < warps; ++w) {
    all.sum += box[w].sum;
    if (MAX) all.max = max_nan(all.max, box[w].max);
  }
  return all;
}

// ------------------------------------------------------------ rows through shared memory

constexpr int RING_WARPS = 16;
constexpr int RING_THREADS = RING_WARPS * 32;
constexpr int RING_MAX_STAGES = 32;   // of all teams
constexpr uint32_t RING_BYTES = 208 * 1024;

// Where a team stands in its rows: those of a CTA go to its teams in turn.
struct RingRows {
  int64_t first, step, count;
};
__device__ __forceinline__ RingRows ring_rows(int64_t rows, int teams, int which) {
  RingRows r;
  r.step = static_cast<int64_t>(gridDim.x) * teams;
  r.first = blockIdx.x + static_cast<int64_t>(which) * gridDim.x;
  r.count = which < teams && r.first < rows ? (rows - r.first + r.step - 1) / r.step : 0;
  return r;
}

// A bounded wait without a call (a call's conventions would spill the sums that
// live across it) and, at first, without the slow global timer.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_test_wait(bar, parity); ++it) {
    if (it & 1023) continue;
    if (*wd.abort) return false;
    if (t0 == 0) t0 = global_timer_ns();
    if (global_timer_ns() - t0 > wd.limit_ns) {
      *wd.abort = 1;
      atomicExch(wd.status, STATUS_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Barrier `id` of `threads` threads; whether `ok` holds for all of them.
__device__ __forceinline__ bool team_sync(int id, int threads, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "r"(id), "r"(threads)
      : "memory");
  return all != 0;
}

// The sum over a team of a value a thread, in every thread, in a fixed order.
// `ok` is false after it unless it was true in all of them: the team's warps give
// up together. What the team's threads read before it, they have read: one of them may
// then fill that memory anew. `box`: a slot for each warp of the CTA, not used again before
// the next sum but one.
__device__ __forceinline__ float ring_sum(float sum, int which, int team, float* box, bool* ok) {
  const int warps = team / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (warps == 1) {
    __syncwarp();   // the shuffles alone order no memory
    return sum;
  }
  if (lane == 0) box[threadIdx.x / 32] = sum;
  *ok = team_sync(1 + which, team, *ok);
  sum = (lane & 15) < warps ? box[which * warps + (lane & 15)] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// ------------------------------------------------------------ forward

struct NormParams {
  const void *x, *residual, *weight;   // residual may be NULL
  void *h, *y;                         // h may be NULL
  float *rstd, *scales;                // may be NULL (scales iff Q == 0)
  int64_t ldx, ldr, ldh, ldy;          // elements between rows
  int64_t rows;
  int cols;
  int team;                            // threads a row: 32 (blockDim / 32 rows a block), or all
  float eps;
  Dropout drop;
};

// Blocks of `most` threads that an SM has to hold, which bounds their registers: so that
// another row's loads are under way while one waits for its sum. On the general path in
// 16 bits two rows of 512 threads (8192 x 8191 bf16: 164 us, with one of them 270).
constexpr int rows_at_once(bool any, int bytes, int vpt, int most) {
  return most == 256 ? (bytes == 2 ? 3 : 2) : any && bytes == 2 && vpt == 2 ? 2 : 1;
}

// One row a team. Q: 0 y has the type of x; 1 e4m3 with one scale a row; 2
// e4m3 with a scale for each 128 columns.
template <typename T, Path PATH, int VPT, int MOST, int Q>
__global__ void __launch_bounds__(MOST, rows_at_once(PATH == ANY, sizeof(T), VPT, MOST))
    add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ SumMax box[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
  if (row >= p.rows) return;   // only whole warps, and only where a team is a warp
  const Row<T> x = row_of<T>(p.x, row, p.rows, p.ldx), res = row_of<T>(p.residual, row, p.rows, p.ldr),
               weight = row_of<T>(p.weight, 0, 1, 0);
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  constexpr bool WHOLE = PATH != ANY;

  if constexpr (!WHOLE) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (k * team + t) * GROUP;
      if (c < cols) {
        prefetch_group(x, c);
        if (p.residual) prefetch_group(res, c);
      }
    }
  }
  Raw<T> xr[VPT] = {}, rr[VPT], wr[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      xr[k] = load_group<WHOLE>(x, g * GROUP, cols);
      if (p.residual) rr[k] = load_group<WHOLE>(res, g * GROUP, cols);
      wr[k] = load_group<WHOLE>(weight, g * GROUP, cols);
    }
  }
  const uint64_t seed = p.drop.rng[0];
  const uint64_t first = p.drop.rng[1] + static_cast<uint64_t>(row) * groups;
  float v[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k) unpack(xr[k], v[k]);
  if (PATH == DROP || (PATH == ANY && p.drop.on)) {
    constexpr int PAIR = VPT < 2 ? VPT : 2;   // generators side by side; more would cost registers
#pragma unroll
    for (int k = 0; k < VPT; k += PAIR) {
      uint64_t counter[PAIR];
#pragma unroll
      for (int j = 0; j < PAIR; ++j) counter[j] = first + (k + j) * team + t;
      drop_groups(p.drop, seed, counter, reinterpret_cast<float(&)[PAIR][GROUP]>(v[k]));
    }
  }
  SumMax s = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    if (g < groups) {
      float w[GROUP];
      if (Q == 1) unpack(wr[k], w);
      if (p.residual) {
        float r[GROUP];
        unpack(rr[k], r);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) v[k][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        s.sum = fmaf(v[k][i], v[k][i], s.sum);
        if (Q == 1) s.max = max_nan(s.max, fabsf(v[k][i] * w[i]));
      }
    }
    if (p.h && (PATH == ANY || g < groups))
      store_group<WHOLE>(static_cast<T*>(p.h) + row * p.ldh, g * GROUP, cols, t, team, pack<T>(v[k]));
  }
  s = reduce_team<Q == 1>(s, team / 32, box);
  // r of the unrounded h, in 32 bits
  const float r = rsqrtf(s.sum / static_cast<float>(cols) + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = r;
  // Q == 1: max |y| = r * max |h * weight|, so one reduction serves both
  float scale = 0.0f;
  if (Q == 1) {
    scale = max_nan(s.max * r / E4M3_MAX, 1.17549435e-38f);
    if (t == 0) p.scales[row] = scale;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = k * team + t;
    float w[GROUP];
    if (g < groups) {
      unpack(wr[k], w);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) v[k][i] = v[k][i] * r * w[i];
    }
    if (Q == 0) {
      if (PATH == ANY || g < groups)
        store_group<WHOLE>(static_cast<T*>(p.y) + row * p.ldy, g * GROUP, cols, t, team, pack<T>(v[k]));
    } else {
      if (Q == 2) {
        // the 16 groups of 128 columns sit on 16 neighbouring lanes
        float m = 0.0f;
        if (g < groups) {
#pragma unroll
          for (int i = 0; i < GROUP; ++i) m = max_nan(m, fabsf(v[k][i]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        scale = max_nan(m / E4M3_MAX, 1.17549435e-38f);
        if ((t & 15) == 0 && g < groups)
          p.scales[row * ((cols + QUANT_GROUP - 1) / QUANT_GROUP) + g / 16] = scale;
      }
      const uint2 out = quotients(v[k], scale);
      if (PATH == ANY || g < groups)
        store_bytes<WHOLE>(static_cast<uint8_t*>(p.y) + row * p.ldy, g * GROUP, cols, t, team,
                           out);
    }
  }
}

struct NormRing {
  NormParams p;
  int stages, teams;    // stages of a team
  uint32_t row_bytes;   // of one matrix
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;      // 3: only the first stages are ever filled
#endif
};

// The forward pass with dropout for many rows of a 16-bit type that lie FAST: as
// the gradient's ring (see there), since the generator's rounds leave the plain
// kernel too few threads on an SM to cover a row's wait (8192 x 8192 bf16: 100 us,
// here 95, 0.84 of the copy rate; 4096 x 8192 fp32, with half the rounds a byte,
// is faster without: 82 against 97). A team has its row in registers at its
// barrier, so the row's own stage is free then.
template <typename T, int VPT>
__global__ void __launch_bounds__(RING_THREADS, 1)
    add_rms_norm_ring_kernel(const __grid_constant__ NormRing q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ float box[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const NormParams& p = q.p;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const int inputs = p.residual ? 2 : 1;
  const uint32_t stage_bytes = inputs * q.row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.teams * q.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    aborted = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x % team, which = threadIdx.x / team;
  const RingRows rows = ring_rows(p.rows, q.teams, which);
  if (rows.count == 0) return;
  const uint32_t stage0 = smem_addr(ring) + which * q.stages * stage_bytes;
  auto full = [&](int s) { return smem_addr(&bars[which * q.stages + s]); };
  auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
    if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
    const int64_t row = rows.first + k * rows.step;
    const uint32_t dst = stage0 + s * stage_bytes;
    mbar_arrive_expect_tx(full(s), stage_bytes);
    bulk_load_1d(dst, static_cast<const T*>(p.x) + row * p.ldx, q.row_bytes, full(s));
    if (p.residual)
      bulk_load_1d(dst + q.row_bytes, static_cast<const T*>(p.residual) + row * p.ldr, q.row_bytes,
                   full(s));
  };
  if (t == 0)
    for (int k = 0; k < q.stages && k < rows.count; ++k) fetch(k, k);
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  Raw<T> wr[VPT] = {};
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (j * team + t < groups) wr[j] = static_cast<const Raw<T>*>(p.weight)[j * team + t];
  int s = 0, turn = 0;
  uint32_t ph = 0;
  int64_t k = 0;
  for (; k < rows.count; ++k, turn ^= 1) {
    const int64_t row = rows.first + k * rows.step;
    uint64_t counter[VPT];
    uint32_t words[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      counter[j] = first + static_cast<uint64_t>(row) * groups + j * team + t;
    philox(counter, seed, words);
    bool ok = __all_sync(0xffffffffu, ring_wait(full(s), ph, wd));
    const uint8_t* stage = ring + (which * q.stages + s) * stage_bytes;
    const Raw<T>* x = reinterpret_cast<const Raw<T>*>(stage) + t;
    const Raw<T>* res = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
    Raw<T>* h = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.h) + row * p.ldh) + t;
    float v[VPT][GROUP];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * team + t < groups) {
        unpack(x[j * team], v[j]);
        drop_by(p.drop, reinterpret_cast<const uint32_t(&)[1][4]>(words[j]),
                reinterpret_cast<float(&)[1][GROUP]>(v[j]));
        if (p.residual) {
          float r[GROUP];
          unpack(res[j * team], r);
#pragma unroll
          for (int i = 0; i < GROUP; ++i) v[j][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) sum = fmaf(v[j][i], v[j][i], sum);
        if (p.h) h[j * team] = pack<T>(v[j]);
      }
    }
    sum = ring_sum(sum, which, team, box[turn], &ok);
    if (!ok) break;
    if (t == 0 && k + q.stages < rows.count) fetch(k + q.stages, s);   // the row is in registers
    const float r = rsqrtf(sum / static_cast<float>(cols) + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r;
    Raw<T>* y = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.y) + row * p.ldy) + t;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * team + t < groups) {
        float w[GROUP];
        unpack(wr[j], w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) v[j][i] = v[j][i] * r * w[i];
        y[j * team] = pack<T>(v[j]);
      }
    }
    if (++s == q.stages) {
      s = 0;
      ph ^= 1;
    }
  }
  // Given up: the copies under way land before the CTA ends.
  if (k < rows.count && t == 0)
    for (int64_t j = k; j < rows.count && j < k + q.stages; ++j)
      wait_drain(full(static_cast<int>(j % q.stages)), static_cast<uint32_t>(j / q.stages) & 1);
}

// ------------------------------------------------------------ backward

struct NormGradParams {
  const void *dy, *dh, *h, *weight;    // dh may be NULL
  const float* rstd;
  void *dx, *dres;                     // dres may be NULL
  float* partial;                      // dweight partials, one row of whole groups a block; NULL: no dweight
  int64_t lddy, lddh, ldh, lddx, lddres;
  int64_t rows;
  int cols;
  int team;
  Dropout drop;
};

// A block's row of dweight partials: the teams' shares added in the teams' order.
// `box`, for more than one team: a row for each of them, the groups' lower halves
// before the upper ones, so that a warp's 16-byte accesses meet no bank twice. (The
// teams adding to one row in turn took a barrier each: gradient of 16384 x 1024 26.5 us instead of 23.)
template <int VPT>
__device__ __forceinline__ void leave_partial(const float (&acc)[VPT][GROUP], float* box, float* partial,
                                              int groups, int team, int teams, int which, int t) {
  float4* out = reinterpret_cast<float4*>(partial) + static_cast<size_t>(blockIdx.x) * 2 * groups;
  float4* mine = teams == 1 ? out : reinterpret_cast<float4*>(box) + which * 2 * groups;
  const int apart = teams == 1 ? 2 : 1, upper = teams == 1 ? 1 : groups;
  if (which < teams) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g >= groups) continue;
      const float(&a)[GROUP] = acc[k];
      mine[apart * g] = make_float4(a[0], a[1], a[2], a[3]);
      mine[apart * g + upper] = make_float4(a[4], a[5], a[6], a[7]);
    }
  }
  if (teams == 1) return;
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * groups; j += blockDim.x) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int v = 0; v < teams; ++v) {
      const float4 a = reinterpret_cast<const float4*>(box)[v * 2 * groups + j];
      s.x += a.x;
      s.y += a.y;
      s.z += a.z;
      s.w += a.w;
    }
    out[j < groups ? 2 * j : 2 * (j - groups) + 1] = s;
  }
}

// Persistent: a team takes rows blockIdx * teams + team, + all teams of the
// grid, and keeps its columns' share of dweight in registers; a block leaves
// one partial row, and dweight_kernel adds those in block order. So dweight
// has the same bits on every run, whatever the timing.
template <typename T, Path PATH, int VPT, int MOST>
__global__ void __launch_bounds__(MOST, 1)
    add_rms_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ SumMax box[2][32];
  extern __shared__ __align__(16) float share[];   // where a team is a warp: their shares of dweight
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = p.team, t = threadIdx.x % team, teams = blockDim.x / team;
  const int cols = p.cols, groups = (cols + GROUP - 1) / GROUP;
  constexpr bool WHOLE = PATH != ANY;
  const Row<T> weight = row_of<T>(p.weight, 0, 1, 0);
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  float acc[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP; ++i) acc[k][i] = 0.0f;

  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * teams + threadIdx.x / team; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * teams, turn ^= 1) {
    const Row<T> dy = row_of<T>(p.dy, row, p.rows, p.lddy), h = row_of<T>(p.h, row, p.rows, p.ldh),
                 dh = row_of<T>(p.dh, row, p.rows, p.lddh);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int c = (k * team + t) * GROUP;
        if (c < cols) {
          prefetch_group(dy, c);
          prefetch_group(h, c);
          if (p.dh) prefetch_group(dh, c);
        }
      }
    }
    Raw<T> yr[VPT], hr[VPT], dr[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        yr[k] = load_group<WHOLE>(dy, g * GROUP, cols);
        hr[k] = load_group<WHOLE>(h, g * GROUP, cols);
        if (p.dh) dr[k] = load_group<WHOLE>(dh, g * GROUP, cols);
      }
    }
    const float r = p.rstd[row];
    SumMax s = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], n[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], n);
        unpack(load_group<WHOLE>(weight, g * GROUP, cols), w);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          const float ni = n[i] * r;
          acc[k][i] = fmaf(a[i], ni, acc[k][i]);
          s.sum = fmaf(a[i] * w[i], ni, s.sum);
        }
      }
    }
    const float c = reduce_team<false>(s, team / 32, box[turn]).sum / static_cast<float>(cols);
    const float rc = r * c;
    float d[VPT][GROUP];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (g < groups) {
        float a[GROUP], n[GROUP], w[GROUP];
        unpack(yr[k], a);
        unpack(hr[k], n);
        unpack(load_group<WHOLE>(weight, g * GROUP, cols), w);
        unpack(dr[k], d[k]);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) d[k][i] = fmaf(r, a[i] * w[i] - n[i] * rc, d[k][i]);
      }
      if (p.dres && (PATH == ANY || g < groups))
        store_group<WHOLE>(static_cast<T*>(p.dres) + row * p.lddres, g * GROUP, cols, t, team,
                           pack<T>(d[k]));
    }
    if (PATH == DROP || (PATH == ANY && p.drop.on)) {
      uint64_t counter[VPT];
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        counter[k] = first + static_cast<uint64_t>(row) * groups + k * team + t;
      drop_groups(p.drop, seed, counter, d);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int g = k * team + t;
      if (PATH == ANY || g < groups)
        store_group<WHOLE>(static_cast<T*>(p.dx) + row * p.lddx, g * GROUP, cols, t, team, pack<T>(d[k]));
    }
  }
  if (p.partial) leave_partial(acc, share, p.partial, groups, team, teams, threadIdx.x / team, t);
}

// The same for many rows that lie FAST: the rows come through a ring in shared
// memory by bulk copies, so that the next rows are on their way while a team
// waits for its row's sum (loaded straight into registers the rows of an SM stop
// at each such wait: 8192 x 8192 bf16 took 124 us, with dropout 171, against 87
// and 107: 0.91 and 0.93 of the copy rate). RING_WARPS warps form teams of `team`
// threads; row k of a CTA goes to its team k % teams, each of which has its own
// stages. There is no producer warp: a team's barrier of a row says that all of it
// is done with the row before, whose stage one thread then fills again. (With such
// a warp the CTA's 17 warps count as 20, which leaves 96 registers a thread instead
// of 128, and four groups a thread spill.) Both passes over a row read it from the
// ring: holding it in registers in between cost more (130 us) than the second
// reading.
struct NormGradRing {
  NormGradParams p;
  int stages, teams;    // stages of a team
  uint32_t row_bytes;   // of one matrix
  uint32_t* status;
  unsigned long long timeout_ns;
#ifdef GEMM_WS_DEBUG
  int debug_fault;      // 3: only the first stages are ever filled
#endif
};

template <typename T, bool ON, int VPT>
__global__ void __launch_bounds__(RING_THREADS, 1)
    add_rms_norm_grad_ring_kernel(const __grid_constant__ NormGradRing q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[RING_MAX_STAGES];
  __shared__ float box[2][RING_WARPS];
  __shared__ uint32_t aborted;
  const NormGradParams& p = q.p;
  const int cols = p.cols, groups = cols / GROUP, team = p.team;
  const int inputs = p.dh ? 3 : 2;
  const uint32_t stage_bytes = inputs * q.row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.teams * q.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    aborted = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const Watchdog wd{&aborted, q.status, q.timeout_ns};
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x % team, which = threadIdx.x / team;
  const RingRows rows = ring_rows(p.rows, q.teams, which);

  Pair acc[VPT][GROUP / 2];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP / 2; ++i) acc[k][i] = 0;

  if (rows.count > 0) {
    const uint32_t stage0 = smem_addr(ring) + which * q.stages * stage_bytes;
    auto full = [&](int s) { return smem_addr(&bars[which * q.stages + s]); };
    // One thread of the team fetches row k into stage s.
    auto fetch = [&](int64_t k, int s) {
#ifdef GEMM_WS_DEBUG
      if (q.debug_fault == 3 && k >= q.stages) return;   // injected fault: the row never comes
#endif
      const int64_t row = rows.first + k * rows.step;
      const uint32_t dst = stage0 + s * stage_bytes;
      mbar_arrive_expect_tx(full(s), stage_bytes);
      bulk_load_1d(dst, static_cast<const T*>(p.dy) + row * p.lddy, q.row_bytes, full(s));
      bulk_load_1d(dst + q.row_bytes, static_cast<const T*>(p.h) + row * p.ldh, q.row_bytes, full(s));
      if (p.dh)
        bulk_load_1d(dst + 2 * q.row_bytes, static_cast<const T*>(p.dh) + row * p.lddh, q.row_bytes,
                     full(s));
    };
    if (t == 0)
      for (int k = 0; k < q.stages && k < rows.count; ++k) fetch(k, k);
    const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
    Raw<T> wr[VPT] = {};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (j * team + t < groups) wr[j] = static_cast<const Raw<T>*>(p.weight)[j * team + t];
    int s = 0, turn = 0, before = q.stages - 1;   // this row's stage, and the one before's
    uint32_t ph = 0;
    float next_r = p.rstd[rows.first];
    int64_t k = 0;
    for (; k < rows.count; ++k, turn ^= 1) {
      const int64_t row = rows.first + k * rows.step;
      const float r = next_r;
      if (k + 1 < rows.count) next_r = p.rstd[row + rows.step];
      // The mask needs nothing of the row: its rounds fill the wait for it.
      uint32_t words[VPT][4];
      if (ON) {
        uint64_t counter[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          counter[j] = first + static_cast<uint64_t>(row) * groups + j * team + t;
        philox(counter, seed, words);
      }
      bool ok = __all_sync(0xffffffffu, ring_wait(full(s), ph, wd));
      const uint8_t* stage = ring + (which * q.stages + s) * stage_bytes;
      const Raw<T>* dy = reinterpret_cast<const Raw<T>*>(stage) + t;
      const Raw<T>* h = reinterpret_cast<const Raw<T>*>(stage + q.row_bytes) + t;
      const Raw<T>* dh = reinterpret_cast<const Raw<T>*>(stage + 2 * q.row_bytes) + t;
      // acc += dy h r, and the sum of dy weight h
      const Pair r2 = pair_of(r, r);
      Pair sums = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j * team + t < groups) {
          Pair a[GROUP / 2], n[GROUP / 2], w[GROUP / 2];
          unpack(dy[j * team], a);
          unpack(h[j * team], n);
          unpack(wr[j], w);
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            const Pair an = mul2(a[i], n[i]);
            acc[j][i] = fma2(an, r2, acc[j][i]);
            sums = fma2(an, w[i], sums);
          }
        }
      }
      const float sum =
          ring_sum(values_of(sums).x + values_of(sums).y, which, team, box[turn], &ok);
      if (!ok) break;
      // The whole team has been in the sum, so it has done with the row before.
      if (t == 0 && k > 0 && k - 1 + q.stages < rows.count) fetch(k - 1 + q.stages, before);
      // dres = dh + r dy weight - h r^2 mean(dy weight h r)
      const float m = -r * r * (r * sum / static_cast<float>(cols));
      const Pair m2 = pair_of(m, m);
      Raw<T>* dres = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dres) + row * p.lddres) + t;
      Raw<T>* dx = reinterpret_cast<Raw<T>*>(static_cast<T*>(p.dx) + row * p.lddx) + t;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j * team + t < groups) {
          Pair a[GROUP / 2], n[GROUP / 2], w[GROUP / 2], e[GROUP / 2];
          unpack(dy[j * team], a);
          unpack(h[j * team], n);
          unpack(wr[j], w);
          Raw<T> dr = {};
          if (p.dh) dr = dh[j * team];
          unpack(dr, e);
          float d[1][GROUP];
#pragma unroll
          for (int i = 0; i < GROUP / 2; ++i) {
            e[i] = fma2(n[i], m2, fma2(mul2(a[i], w[i]), r2, e[i]));
            d[0][2 * i] = values_of(e[i]).x;
            d[0][2 * i + 1] = values_of(e[i]).y;
          }
          if (p.dres) dres[j * team] = pack<T>(d[0]);
          if (ON) drop_by(p.drop, reinterpret_cast<const uint32_t(&)[1][4]>(words[j]), d);
          dx[j * team] = pack<T>(d[0]);
        }
      }
      before = s;
      if (++s == q.stages) {
        s = 0;
        ph ^= 1;
      }
    }
    // Given up: the copies under way land before the CTA ends.
    if (k < rows.count && t == 0)
      for (int64_t j = k; j < rows.count && j < k + q.stages - (k > 0); ++j)
        wait_drain(full(static_cast<int>(j % q.stages)), static_cast<uint32_t>(j / q.stages) & 1);
  }
  if (!p.partial) return;
  float mine[VPT][GROUP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < GROUP / 2; ++i) {
      mine[k][2 * i] = values_of(acc[k][i]).x;
      mine[k][2 * i + 1] = values_of(acc[k][i]).y;
    }
  __syncthreads();   // all teams have done with the ring
  static_assert(RING_THREADS * VPT * GROUP * sizeof(float) <= RING_BYTES, "the teams' rows fit the ring");
  leave_partial(mine, reinterpret_cast<float*>(ring), p.partial, groups, team, q.teams, which, t);
}

constexpr int DW_QUADS = 4, DW_COLS = 4 * DW_QUADS, DW_LANES = 128;   // a block's columns; partial rows in flight
constexpr int DW_THREADS = DW_QUADS * DW_LANES;

struct DweightParams {
  const float* partial;
  int blocks, cols, pitch;
  void* dweight;
};

// dweight[c] = the sum of the blocks' partial rows, in a fixed order. A thread has four
// columns of every 128th row, eight of them in flight at once. There are 152 rows from a ring
// (two a thread), and up to 2432 (19 a thread) where the blocks are smallest: of 64 threads,
// of unaligned rows of 257 to 512 columns.
template <typename T>
__global__ void __launch_bounds__(DW_THREADS)
    dweight_kernel(const __grid_constant__ DweightParams p) {
  __shared__ float box[DW_THREADS / 32][DW_COLS];
  grid_dependency_wait();
  grid_launch_dependents();
  const int x = threadIdx.x % DW_QUADS, lane = threadIdx.x / DW_QUADS;
  const int quads = p.pitch / 4, quad = blockIdx.x * DW_QUADS + x;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (quad < quads) {
    const float4* rows = reinterpret_cast<const float4*>(p.partial) + quad;
#pragma unroll 8
    for (int b = lane; b < p.blocks; b += DW_LANES) {
      const float4 a = rows[static_cast<size_t>(b) * quads];
      s.x += a.x;
      s.y += a.y;
      s.z += a.z;
      s.w += a.w;
    }
  }
#pragma unroll
  for (int o = DW_QUADS; o < 32; o *= 2) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
  }
  if (threadIdx.x % 32 < DW_QUADS) {
    float* to = box[threadIdx.x / 32] + 4 * x;
    to[0] = s.x;
    to[1] = s.y;
    to[2] = s.z;
    to[3] = s.w;
  }
  __syncthreads();
  const int c = blockIdx.x * DW_COLS + threadIdx.x;
  if (threadIdx.x < DW_COLS && c < p.cols) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < DW_THREADS / 32; ++w) sum += box[w][threadIdx.x];
    static_cast<T*>(p.dweight)[c] = round_to(sum, T());
  }
}

// ------------------------------------------------------------ dropout alone

struct DropoutParams {
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int64_t rows;
  int cols;
  int64_t groups;      // FLAT: of the whole matrix; else of a row
  int row_threads;     // not FLAT: threads of a row, a power of two
  Dropout drop;
};

constexpr int DROP_THREADS = 256, DROP_VPT = 2;

// FLAT: rows follow one another without gaps in whole groups, so the matrix is
// one run of groups and no row has to be found. ON: p > 0.
template <typename T, bool ON>
__global__ void __launch_bounds__(DROP_THREADS) dropout_flat_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (DROP_THREADS * DROP_VPT) + threadIdx.x;
  Raw<T> raw[DROP_VPT] = {};
  float v[DROP_VPT][GROUP];
  uint64_t counter[DROP_VPT];
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) raw[k] = static_cast<const Raw<T>*>(p.x)[g];
    counter[k] = first + g;
  }
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) unpack(raw[k], v[k]);
  if (ON) drop_groups(p.drop, seed, counter, v);
#pragma unroll
  for (int k = 0; k < DROP_VPT; ++k) {
    const int64_t g = base + k * DROP_THREADS;
    if (g < p.groups) static_cast<Raw<T>*>(p.y)[g] = pack<T>(v[k]);
  }
}

// Any rows: row_threads threads walk one, DROP_THREADS / row_threads rows a block.
template <typename T>
__global__ void __launch_bounds__(DROP_THREADS) dropout_rows_kernel(const __grid_constant__ DropoutParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t seed = p.drop.rng[0], first = p.drop.rng[1];
  const int team = p.row_threads, t = threadIdx.x % team;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (DROP_THREADS / team) + threadIdx.x / team;
  const bool there = row < p.rows;
  const Row<T> x = row_of<T>(p.x, there ? row : 0, p.rows, p.ldx);
  T* y = static_cast<T*>(p.y) + (there ? row : 0) * p.ldy;
  const int groups = static_cast<int>(p.groups);
  for (int g0 = 0; g0 < groups; g0 += team) {   // whole warps stay together for the stores
    const int g = g0 + t;
    const bool mine = there && g < groups;
    Raw<T> raw = {};
    if (mine) raw = load_group<false>(x, column_of(g, groups, p.cols), p.cols);
    float v[1][GROUP];
    unpack(raw, v[0]);
    const uint64_t counter[1] = {first + static_cast<uint64_t>(row) * groups + g};
    if (p.drop.on) drop_groups(p.drop, seed, counter, v);
    store_group<false>(y, column_of(mine ? g : groups, groups, p.cols), p.cols, t, team, pack<T>(v[0]));
  }
}

}  // namespace gws
