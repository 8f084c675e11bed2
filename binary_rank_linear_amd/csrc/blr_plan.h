// A plan's groups of positions (internal; no device header, so that the host's
// tests can compile it by itself).
#pragma once

namespace blr {

// An offset's place in a plan of M positions, whatever it holds.
constexpr int plan_at(int offset, int M) { return offset < 0 ? 0 : offset > M ? M : offset; }

// Positions of the group between two offsets. Both are brought into [0, M]
// before they are subtracted, so that neither order nor size of them can
// overflow the count or lead outside the plan.
constexpr int plan_rows(int lo, int hi, int M) {
    return plan_at(hi, M) > plan_at(lo, M) ? plan_at(hi, M) - plan_at(lo, M) : 0;
}

}  // namespace blr
