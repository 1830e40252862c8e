// Layout of the paged block-quantized key / value cache (tq_cache_write,
// tq_cache_read, tq_tree_attention).
//
// A cache buffer is [page][kv head] chunks of page_size tokens; a chunk is
// all its codes, then all its fp16 scales.  Codes are unsigned: Q8_0 code +
// 128 in a byte, Q4_0 the nibble 0..15 (code + 8).  The orders inside a
// chunk are those in which one lane of the attention's 16x16x32 fp16 matrix
// instructions wants its operand, so that codes go from memory to the matrix
// cores through registers alone:
//
//   K codes  [token][D]: lane group g (0..3) of an instruction holds elements
//            8g..8g+7 of a 32-element block s.  Eight elements are one piece
//            (8 bytes Q8_0, 4 bytes Q4_0), and the pieces one lane needs lie
//            together in up to 16 bytes (k_piece_off).
//   K scales [token][D / 32].
//   V codes  [token / 4][column][token % 4]: 4 tokens of one element (Q8_0:
//            column = element) or of an element pair (Q4_0: column c holds
//            elements 2c, 2c + 1 in the low / high nibble) in a dword, because
//            the product with the probabilities contracts over tokens.
//   V scales [D / 32][token].
//
// Nibbles and bytes are placed so that the pairs that (w >> 4j) & 0x000f000f
// picks out are neighbours in the operand: element i of a Q4_0 K piece is
// nibble k4_shift(i), token t of a Q4_0 V dword is byte v4_byte(t).
#pragma once

#include <stdint.h>

#include "tiledq.h"

namespace tq {

constexpr bool cache_type_ok(int ct) { return ct == TQ_Q8_0 || ct == TQ_Q4_0; }
constexpr bool cache_dim_ok(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }
constexpr bool cache_page_ok(int64_t P) { return P >= 16 && P <= 1024 && (P & (P - 1)) == 0; }

// Bytes of the codes of one token of one head, and of one [page][head] chunk.
constexpr int64_t token_code_bytes(int ct, int64_t D) { return ct == TQ_Q8_0 ? D : D / 2; }
constexpr int64_t chunk_bytes(int ct, int64_t D, int64_t P)
{
    return P * (token_code_bytes(ct, D) + D / 16);
}

// Byte offset, within a token's K codes, of the piece of block s for lane
// group g.  One lane's pieces of consecutive blocks are gathered into 16
// bytes where D gives whole 16-byte groups, into D / 8 bytes (Q4_0) or
// single 8-byte pieces (Q8_0, D = 96) otherwise.
template <int CT, int D>
__host__ __device__ constexpr int k_piece_off(int s, int g)
{
    if constexpr (CT == TQ_Q8_0)
        return D % 64 == 0 ? ((s >> 1) * 4 + g) * 16 + (s & 1) * 8 : s * 32 + g * 8;
    else
        return D % 128 == 0 ? ((s >> 2) * 4 + g) * 16 + (s & 3) * 4 : g * (D / 8) + s * 4;
}

// Bit position of element i (0..7) in a Q4_0 K piece.
__host__ __device__ constexpr int k4_shift(int i)
{
    const int f = i >> 1, h = i & 1;
    return 8 * (2 * h + (f >> 1)) + 4 * (f & 1);
}

// Byte of token t (0..3) in a Q4_0 V dword.
__host__ __device__ constexpr int v4_byte(int t) { return ((t & 1) << 1) | (t >> 1); }

}  // namespace tq
