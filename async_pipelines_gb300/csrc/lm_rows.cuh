// Rows of a matrix in the registers of a team of threads, 8 columns (a "group", 16
// bytes of a 16-bit type) at a time: loads and stores of aligned and unaligned
// rows, conversions, sums over a team, and the ring in shared memory that rows come
// through. What the kernels of lm_norm_kernel.cuh and lm_block_kernel.cuh share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx.cuh"
#include "watchdog.cuh"

namespace gws {

constexpr int GROUP = 8;                 // columns of a group
constexpr int QUANT_GROUP = 128;         // columns of one scale (Q == 2)
constexpr int MAX_VPT = 4;               // groups a thread holds
constexpr float E4M3_MAX = 448.0f;       // largest finite e4m3

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

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
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

// The 8-bit integers nearest to v / scale (halves to even), lowest column first, |v| < 127.5 scale;
// zeros where scale is NaN. As the quotients above: put between two products, and divided only
// where those round differently. A sum with 1.5 * 2^23 leaves the rounded integer in the
// sum's low bits, without the conversion unit's quarter rate.
__device__ __forceinline__ uint2 int8_quotients(const float (&v)[GROUP], float scale) {
  constexpr float SHIFT = 12582912.0f;
  auto bytes = [](const float (&q)[GROUP]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __byte_perm(__float_as_uint(q[4 * i]), __float_as_uint(q[4 * i + 1]), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(q[4 * i + 2]), __float_as_uint(q[4 * i + 3]), 0x0040);
      w[i] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(w[0], w[1]);
  };
  if (!(scale == scale)) return make_uint2(0, 0);
  const float inv = 1.0f / scale;
  auto times = [&](float factor) {
    const Pair f = pair_of(factor, factor), shift = pair_of(SHIFT, SHIFT);
    float q[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; i += 2) {
      const float2 two = values_of(fma2(pair_of(v[i], v[i + 1]), f, shift));
      q[i] = two.x;
      q[i + 1] = two.y;
    }
    return bytes(q);
  };
  const uint2 least = times(inv * (1.0f - 0x1p-22f)), most = times(inv * (1.0f + 0x1p-22f));
  if (least.x == most.x && least.y == most.y) return least;
  float q[GROUP];
#pragma unroll
  for (int i = 0; i < GROUP; ++i) q[i] = __fadd_rn(__fdiv_rn(v[i], scale), SHIFT);
  return bytes(q);
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

// The same for a sum and a maximum.
__device__ __forceinline__ SumMax ring_sum_max(SumMax v, int which, int team, SumMax* box, bool* ok) {
  const int warps = team / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    v.max = max_nan(v.max, __shfl_xor_sync(0xffffffffu, v.max, o));
  }
  if (warps == 1) {
    __syncwarp();
    return v;
  }
  if (lane == 0) box[threadIdx.x / 32] = v;
  *ok = team_sync(1 + which, team, *ok);
  v = (lane & 15) < warps ? box[which * warps + (lane & 15)] : SumMax{0.0f, 0.0f};
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    v.max = max_nan(v.max, __shfl_xor_sync(0xffffffffu, v.max, o));
  }
  return v;
}

// ------------------------------------------------------------ sums over the rows

// A block's row of partial sums by columns: the teams' shares added in the teams' order.
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

constexpr int DW_QUADS = 4, DW_COLS = 4 * DW_QUADS, DW_LANES = 128;   // a block's columns; partial rows in flight
constexpr int DW_THREADS = DW_QUADS * DW_LANES;

// put(c, the sum of column c over the blocks' partial rows), in a fixed order, for block
// number `block` of the columns. A thread has four columns of every 128th row, eight of them in flight at
// once. There are 152 rows from a ring (two a thread), and most where the blocks are smallest, for unaligned rows of
// 257 to 512 columns: of add_rms_norm up to 2432, from blocks of 64 threads (19 a thread), of block_norm 4864,
// from blocks of one warp (38; 16384 x 511 bf16 104 us in all).
template <typename Put>
__device__ __forceinline__ void column_sums(const float* partial, int block, int blocks, int cols,
                                            int pitch, Put put) {
  __shared__ float box[DW_THREADS / 32][DW_COLS];
  const int x = threadIdx.x % DW_QUADS, lane = threadIdx.x / DW_QUADS;
  const int quads = pitch / 4, quad = block * DW_QUADS + x;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (quad < quads) {
    const float4* rows = reinterpret_cast<const float4*>(partial) + quad;
#pragma unroll 8
    for (int b = lane; b < blocks; b += DW_LANES) {
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
  const int c = block * DW_COLS + threadIdx.x;
  if (threadIdx.x < DW_COLS && c < cols) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < DW_THREADS / 32; ++w) sum += box[w][threadIdx.x];
    put(c, sum);
  }
}

}  // namespace gws
