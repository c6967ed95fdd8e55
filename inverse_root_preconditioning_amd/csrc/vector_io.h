// Vector access to tensors of any alignment, and reductions over small groups
// of lanes: shared by the kernels of the operators beside the preconditioner.
#pragma once

#include "common.h"

namespace shp {

// Global-memory access (see ldg, stg) for a vector at an address aligned to ALIGN bytes only (global
// memory takes vector accesses at any element's address).
template <class V, int ALIGN>
__device__ __forceinline__ V ldg_any(const void* p) {
  typedef V U __attribute__((aligned(ALIGN)));
  return *(const __attribute__((address_space(1))) U*)p;
}
template <class V, int ALIGN>
__device__ __forceinline__ void stg_any(void* p, const V& v) {
  typedef V U __attribute__((aligned(ALIGN)));
  *(__attribute__((address_space(1))) U*)p = v;
}

// The same for data that is read or written once: not kept in the caches.
template <class V, int ALIGN>
__device__ __forceinline__ V ldg_once(const void* p) {
  typedef V U __attribute__((aligned(ALIGN)));
  return __builtin_nontemporal_load((const __attribute__((address_space(1))) U*)p);
}
template <class V, int ALIGN>
__device__ __forceinline__ void stg_once(void* p, const V& v) {
  typedef V U __attribute__((aligned(ALIGN)));
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) U*)p);
}

// Largest of v over groups of 4, 8 or 16 consecutive lanes, in every lane.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  static_assert(LANES == 4 || LANES == 8 || LANES == 16, "lanes of a group");
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));  // quad_perm 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));  // quad_perm 2 3 0 1
  if constexpr (LANES >= 8)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror
  if constexpr (LANES == 16)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // row_mirror
  return v;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t abs_halves(uint32_t a) { return a & 0x7fff7fffu; }

// V consecutive elements of a row: bf16, two a word, or fp32 bits.
template <bool BF16, int V>
struct Piece {
  static constexpr int kElems = V, kWords = BF16 ? V / 2 : V;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  Words w;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    if constexpr (BF16) {
      w = ldg_any<Words, 2>(static_cast<const uint16_t*>(x) + at);
    } else {
      w = ldg_any<Words, 4>(static_cast<const float*>(x) + at);
    }
  }
  __device__ __forceinline__ void load_at(const void* row, uint32_t col) {
    w = ldg_any<Words, BF16 ? 2 : 4>(static_cast<const uint8_t*>(row) + col * (BF16 ? 2u : 4u));
  }
  // The same for what is read once.
  __device__ __forceinline__ void load_once(const void* row, uint32_t col) {
    w = ldg_once<Words, BF16 ? 2 : 4>(static_cast<const uint8_t*>(row) + col * (BF16 ? 2u : 4u));
  }
  // Element e + d at e, 0 from V - d on (0 <= d <= V).
  __device__ __forceinline__ void shift_down(uint32_t d) {
    if constexpr (BF16) {
      if (d & 1) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = (w[i] >> 16) | (i + 1 < kWords ? w[i + 1] << 16 : 0u);
      }
    }
#pragma unroll
    for (int b = 1; b < kWords; b *= 2) {
      if (d & (BF16 ? 2 * b : b)) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = i + b < kWords ? w[i + b] : 0u;
      }
    }
    if (d == V) w = (Words)0u;
  }
  // The piece at (row, col) of a matrix whose edge it may cross (or pass), zero
  // outside.  No branch on the lane: V elements that are there, shifted down.
  __device__ __forceinline__ void load_edge(const void* x, int64_t rows, int64_t cols, int64_t ld, int64_t row,
                                            int64_t col) {
    if (cols >= V) {
      const int64_t from = min(col, cols - V);
      const uint32_t d = row < rows ? (uint32_t)min<int64_t>(col - from, V) : (uint32_t)V;
      load(x, min(row, rows - 1) * ld + from);
      shift_down(d);
    } else {
      w = (Words)0u;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (row < rows && col + e < cols) {
          if constexpr (BF16) {
            w[e / 2] |= (uint32_t)ldg(static_cast<const uint16_t*>(x) + row * ld + col + e) << (16 * (e & 1));
          } else {
            w[e] = ldg(static_cast<const uint32_t*>(x) + row * ld + col + e);
          }
        }
      }
    }
  }
  // Bits, as fp32, of the largest magnitude.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max_halves(m, abs_halves(w[i]));
      return max(m & 0xffff0000u, m << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
};

// The V columns from col of a row of `cols`, zero beyond them.  Column numbers
// of 32 bits unsigned: a uniform row and an offset a lane make one address.
template <bool BF16, int V>
__device__ __forceinline__ Piece<BF16, V> load_row(const void* row, uint32_t cols, uint32_t col) {
  Piece<BF16, V> x;
  if (cols % V == 0) {
    x.w = 0u;
    if (col < cols) x.load_at(row, col);
  } else if (cols > V) {
    const uint32_t from = min(col, cols - V);
    x.load_at(row, from);
    x.shift_down(min(col - from, (uint32_t)V));
  } else {
    x.w = 0u;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (col + e < cols) {
        if constexpr (BF16) {
          x.w[e / 2] |= (uint32_t)ldg(static_cast<const uint16_t*>(row) + e) << (16 * (e & 1));
        } else {
          x.w[e] = ldg(static_cast<const uint32_t*>(row) + e);
        }
      }
    }
  }
  return x;
}

template <bool BF16, int V>
__device__ __forceinline__ float elem(const Piece<BF16, V>& x, int e) {
  if constexpr (BF16) {
    return __builtin_bit_cast(float, (e & 1) ? (uint32_t)x.w[e / 2] & 0xffff0000u : (uint32_t)x.w[e / 2] << 16);
  } else {
    return __builtin_bit_cast(float, (uint32_t)x.w[e]);
  }
}

// x rounded to nearest even into those of the V columns from col that are below cols (WHOLE: all are).
template <bool BF16, int V, bool WHOLE = false>
__device__ __forceinline__ void store_row(void* row, uint32_t cols, uint32_t col, const float (&x)[V]) {
  Piece<BF16, V> o;
#pragma unroll
  for (int i = 0; i < o.kWords; ++i) {
    if constexpr (BF16) {
      o.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    } else {
      o.w[i] = __builtin_bit_cast(uint32_t, x[i]);
    }
  }
  typedef typename Piece<BF16, V>::Words Words;
  if (WHOLE || col + V <= cols) {
    stg_once<Words, BF16 ? 2 : 4>(static_cast<uint8_t*>(row) + col * (BF16 ? 2u : 4u), o.w);
  } else if (col < cols) {
    // the elements that are left in halves, quarters, ... of a piece, each stored from its front
    const uint32_t left = cols - col;
    uint8_t* at = static_cast<uint8_t*>(row) + col * (BF16 ? 2u : 4u);
    static_for<3>([&](auto I) __attribute__((always_inline)) {
      constexpr int n = V >> (decltype(I)::value + 1);  // elements, of kBytes
      constexpr int kBytes = n * (BF16 ? 2 : 4);
      if constexpr (n > 0) {
        if (left & n) {
          if constexpr (kBytes >= 4) {
            typedef uint32_t Part __attribute__((ext_vector_type(kBytes / 4)));
            Part q;
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) q[i] = o.w[i];
            stg_any<Part, BF16 ? 2 : 4>(at, q);
#pragma unroll
            for (int i = 0; i + kBytes / 4 < o.kWords; ++i) o.w[i] = o.w[i + kBytes / 4];
          } else {
            stg(reinterpret_cast<uint16_t*>(at), (uint16_t)(uint32_t)o.w[0]);
          }
          at += kBytes;
        }
      }
    });
  }
}

// Address of a row of a matrix of bf16 or fp32 elements.
template <bool BF16>
__device__ __forceinline__ const void* row_at(const void* x, int64_t row, int64_t ld) {
  return static_cast<const uint8_t*>(x) + row * ld * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ void* row_at(void* x, int64_t row, int64_t ld) {
  return static_cast<uint8_t*>(x) + row * ld * (BF16 ? 2 : 4);
}

}  // namespace shp
