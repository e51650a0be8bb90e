// Which dims of a key the lanes of attention's split kernel load, and the dims of
// q that meet them.  Plain integer functions, so that every case can be
// enumerated on the host.
//
// A lane of group g (0 .. 3) holds HDP / 4 dims of a key in loads of up to 16
// bytes.  Of a head narrower than HDP
// - a load whose dims all lie past head_dim takes the row's first ones, and q is
//   zero there;
// - at 4 bits a load of 32 dims can meet the last 16 of a head (head_dim % 32 ==
//   16).  It then starts 16 dims earlier, so that it ends with the row, and q is
//   zero over its first half, which the load before holds.  Such a load is 8-byte
//   aligned, as the rows of such a head are.
#pragma once

namespace gptq {

template <int HDP, int BITS>
struct KeyLanes {
  static constexpr int kWords = HDP * BITS / 128;          // 32-bit words of a key in a lane
  static constexpr int kLoad = kWords < 4 ? kWords : 4;    // words of one load
  static constexpr int kLoads = kWords / kLoad;
  static constexpr int kDims = kLoad * (32 / BITS);        // dims of one load
  static constexpr int kAlign = BITS == 8 ? 16 : 8;        // bytes
  static constexpr int kSteps = HDP / 32;                  // products of 8 dims a lane

  // first dim of load e
  static constexpr int begin(int g, int e, int hd) {
    const int d = g * (HDP / 4) + e * kDims;
    return d >= hd ? 0 : d + kDims > hd ? hd - kDims : d;
  }
  // first of the 8 dims of q in step s, or -1: zeros
  static constexpr int q_dim(int g, int s, int hd) {
    const int e = 8 * s / kDims, d = g * (HDP / 4) + e * kDims;
    if (d >= hd) return -1;
    const int at = begin(g, e, hd) + 8 * s - e * kDims;
    return at < d ? -1 : at;
  }
};

}  // namespace gptq
