// tree_rings.h -- the rings of shared-memory stages of the tree attention
// kernels, and which barrier a tile lands on.  Plain C++: a host test walks them
// in orders that a GPU seldom takes.
//
// A wait by parity means one of two phases, the last or the next: it is right
// only if the phase before the one it waits for is known to be complete.  Two
// roles that take a stage's tiles in turn do not know that of each other, so a
// tile lands on a barrier that one role waits for, phase after phase.
#pragma once

#ifdef __CUDACC__
#define M4Q_HD __host__ __device__
#else
#define M4Q_HD
#endif

namespace m4q {

// attention_few.cu, nc blocks of 16 rows.
struct FewRings {
  int ks, vs;   // K and V stages (Q8_0: decoded tiles)
  int rs;       // Q8_0: slots of raw tiles, K, V, K, ...
  int groups;   // Q8_0: groups of 4 warps that decode K (and V) tiles in turn
};
constexpr FewRings few_rings(int d, bool q8, int nc) {
  return q8 ? FewRings{3, d == 128 ? 3 : 4, d == 64 ? 10 : nc == 1 ? 6 : 5, nc == 1 ? 2 : 1}
            : FewRings{d == 128 ? 3 : 6, d == 128 ? 3 : 6, 0, 1};
}
// Landing barrier of a K (kv 0) or V (1) tile in a raw slot.  With an odd ring a slot
// holds K and V tiles in turn, which different warps decode.
M4Q_HD constexpr int few_raw_bar(int rs, int kv, int slot) { return kv * rs + slot; }
// With two groups of a kind, a group that waits for its stage first knows the slot's
// last tile, the other group's, to have landed: it was decoded before the stage was
// read.
constexpr bool few_groups_ok(const FewRings& r) {
  return r.groups == 1 || (r.rs % 2 == 0 && r.rs / 2 >= r.ks && r.rs / 2 >= r.vs);
}


// attention_tree.cu: two tile teams, each with an MMA issuer of its own, take the
// tiles in turn.
struct RowsRings {
  int ks, vs;   // K and V stages
  int rs;       // Q8_0: slots of raw tiles, K, V, K, ...
  int sb;       // score buffers
};
constexpr RowsRings rows_rings(int d, bool q8) {
  return q8 ? RowsRings{2, 2, d == 128 ? 3 : 8, d == 64 ? 3 : 2} : RowsRings{d == 128 ? 3 : 6, d == 128 ? 2 : 5, 0, d == 64 ? 3 : 2};
}
// Landing barrier of a team's K tile in a stage.  With an odd ring a stage holds the
// teams' tiles in turn, and with two score buffers nothing keeps an issuer from its
// next tile until the other team's last one has landed.  (V has one barrier a stage:
// there a stage is always the same team's, or the third score buffer keeps P V of all
// tiles in order.)
M4Q_HD constexpr int rows_k_bar(int ks, int team, int stage) { return team * ks + stage; }
// Where the halves of a row exchange the maxima of tile g, of rows_max_slots: with a
// third score buffer a half may have its next tile's scores, and write its next
// maximum, before the other has read this one.  It cannot be two tiles ahead: both
// meet once a tile between writing and reading.
M4Q_HD constexpr int rows_max_slots(int sb) { return sb == 3 ? 2 : 1; }
M4Q_HD constexpr int rows_max_slot(int sb, int g) { return sb == 3 ? (g >> 1) & 1 : 0; }

}  // namespace m4q
