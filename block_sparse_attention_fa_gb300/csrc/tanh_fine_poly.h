// tanh_fine_poly.h -- generated by gen_poly.py (Remez minimax of tanh(u)/u in v = u^2, |u| <= 0.75, degree 4 in v, max relative error 5.651e-07).  Do not edit.
#pragma once
namespace fa {
constexpr float kTanhFineC0 = 0.999999463558197f;
constexpr float kTanhFineC1 = -0.3332825005054474f;
constexpr float kTanhFineC2 = 0.13258983194828033f;
constexpr float kTanhFineC3 = -0.050056301057338715f;
constexpr float kTanhFineC4 = 0.01292963232845068f;
constexpr float kTanhFineRange = 0.75f;
}  // namespace fa
