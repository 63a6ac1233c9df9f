// Layout of the residual RMS norm backward's ring of rows (host arithmetic, no CUDA types).
#pragma once

#include <stddef.h>

namespace tpmlp {

constexpr int kBwdSmem = 196608;    // most shared memory of the ring; the teams' sums take 64 KB at most
constexpr int kBwdMaxBlocks = 160;  // dweight partial rows at most (one block an SM)
constexpr int kBwdConsumers = 16;   // warps
constexpr int kBwdMaxD = 256 * 4 * kBwdConsumers;
constexpr int kBwdMaxSlots = 32;

// Rows go to blocks in groups: group g of all is the block's group g / blocks, of which row `in` is the block's row
// n = (g / blocks) group + in; that row is in slot (g / blocks) % slots and belongs to team n % teams.
struct BwdRing {
  int blocks;      // CTAs
  int vt;          // vectors of a thread
  int team_warps, teams;
  int group;       // rows of a slot
  int slots;
  int most;        // groups of the block that has most
  int slot_bytes;  // s, dy and ds of a group
  int smem;
};

// Whether a ring of `slots` slots of `group` rows is safe for a block that takes `groups` of them.  The phase parity of a
// slot's barrier is one bit: a team that waits for a group while the slot's previous group has not landed takes the phase
// before that for its own, reads old rows and frees the slot early, and the producer then re-arms a barrier with copies in
// flight.  So every team with a row in a group must have had one in the slot's previous group: all teams have rows in
// every whole group, or a row `in` of a slot always belongs to the same team, or no slot is used twice.
inline bool bwd_ring_ok(int groups, int group, int slots, int teams) {
  if (group < 1 || slots < 1 || slots > kBwdMaxSlots) return false;
  return groups <= slots || group >= teams || slots * group % teams == 0;
}

// d <= kBwdMaxD, rows >= 1.
inline BwdRing bwd_ring(int rows, int d, int sm_count) {
  BwdRing r{};
  r.blocks = sm_count < kBwdMaxBlocks ? sm_count : kBwdMaxBlocks;
  if (rows < r.blocks) r.blocks = rows;
  r.vt = d <= kBwdMaxD / 2 ? 2 : 4;
  r.team_warps = 1;
  while (32 * r.team_warps * r.vt < d / 8) r.team_warps *= 2;
  r.teams = kBwdConsumers / r.team_warps;
  // groups of about 8 KB a tensor, but one for each block at least
  r.group = 8192 / (2 * d);
  if (r.group > rows / r.blocks) r.group = rows / r.blocks;
  if (r.group < 1) r.group = 1;
  // as many slots as fit (two of the widest row)
  auto fit = [&] {
    const int groups = rows / r.group + (rows % r.group != 0);
    r.slot_bytes = 3 * 2 * d * r.group;
    r.most = groups / r.blocks + (groups % r.blocks != 0);
    r.slots = kBwdSmem / r.slot_bytes;
    if (r.slots > kBwdMaxSlots) r.slots = kBwdMaxSlots;
  };
  fit();
  if (r.slots < r.most && r.group < r.teams) {  // slots are used again: bwd_ring_ok
    while (r.group & (r.group - 1)) r.group &= r.group - 1;  // a power of two, as the teams are
    fit();
    r.slots -= r.slots % (r.teams / r.group);
  }
  if (r.slots > r.most) r.slots = r.most;
  r.smem = r.slots * r.slot_bytes;
  if (r.smem < r.teams * d * 4) r.smem = r.teams * d * 4;
  return r;
}

}  // namespace tpmlp
